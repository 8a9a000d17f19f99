"""Pins of the fp64 definitions of tree-drafted decoding (oracle/tree.py), and the library's host helpers (no GPU)."""
import ctypes
import math
import os
import re
import struct

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_27_gb300 as kvc
import workloads
from oracle import tree


def random_parents(rng, B, T):
    par = np.full((B, T), -1, np.int32)
    for t in range(1, T):
        par[:, t] = rng.integers(0, t, B)
    return par


def test_chain_tree_is_the_causal_multi_token_decode():
    wl = workloads.multi_token_decode(1, [5, 16, 40], 5, Hq=4, Hkv=2)
    masks, depths = tree.tree_masks(np.tile(np.arange(-1, 4, dtype=np.int32), (3, 1)))
    out, _ = tree.tree_attention(wl.q, wl.k_pool, wl.v_pool, wl.block_table, wl.ctx, masks, [5] * 3, wl.scale)
    ref = oracle.decode_multi(wl.q, wl.k_pool, wl.v_pool, wl.block_table, wl.ctx, wl.scale)
    assert np.abs(out - ref).max() < 1e-12
    assert (depths == np.arange(5)).all()


def test_rotation_depends_on_the_distance_alone():
    rng = np.random.default_rng(2)
    freq = 1e4 ** (-np.arange(0, 64, 2) / 64)
    for inter in (False, True):
        x, y = rng.standard_normal((2, 1, 1, 64))
        dots = [float((tree.norm_rotate(x, None, 0, np.array([[p]]) * freq, inter)
                       * tree.norm_rotate(y, None, 0, np.array([[p + 7]]) * freq, inter)).sum()) for p in (0, 3, 100)]
        assert np.ptp(dots) < 1e-10
        assert abs(dots[0] - float((x * tree.norm_rotate(y, None, 0, 7 * freq[None], inter)).sum())) < 1e-12
    z = tree.norm_rotate(x, np.ones(64), 0.0, np.zeros((1, 0)), False)
    assert abs((z * z).mean() - 1) < 1e-12


@pytest.mark.parametrize("distinct", [False, True])
def test_verification_emits_the_targets_distribution(distinct):
    """Two drafted children of the root and the draw, over every combination of a grid of uniforms: the first token
    that the step emits (a kept child's or the drawn one) is distributed as the target's row."""
    V, n = 3, 60
    p, q = np.array([0.2, 0.5, 0.3]), np.array([0.5, 0.3, 0.2])
    rows = lambda r: np.stack([r] * 3)  # noqa: E731
    grid = (np.arange(n) + 0.5) / n
    mass = np.zeros(V)
    for a in range(V):
        for b in range(V):
            if distinct and a == b:
                continue
            weight = q[a] * (q[b] / (1 - q[a]) if distinct else q[b])  # how often the draft gives these two
            tokens, parents = [0, a, b], [-1, 0, 0]
            for u1 in grid:
                for u2 in grid:
                    for u0 in grid[::6]:
                        path, nxt = tree.verify(rows(p), rows(q), tokens, parents, [u0, u1, u2], distinct)
                        emitted = tokens[path[1]] if len(path) > 1 else nxt
                        mass[emitted] += weight / (n * n * len(grid[::6]))
    # a kept or refused trial is off by at most one grid step per uniform
    assert np.abs(mass - p).max() < 2.0 / n + 1.0 / len(grid[::6]) * 0.3, mass


def test_commit_moves_the_path_and_nothing_else():
    rng = np.random.default_rng(3)
    pool = rng.standard_normal((2, 6, 2, 16, 4))
    before = pool.copy()
    table = np.array([[4, 1, 0]])
    new = tree.commit([pool], table, [40], [9], [[0, 1, 4, 8]], [4])
    rows = lambda a, n: tree.rows_of(a, table[0], n)  # noqa: E731
    assert new[0] == 40 - 9 + 4
    for lay in range(2):
        old, got = rows(before[lay], 40), rows(pool[lay], 40)
        assert (got[:33] == old[:33]).all()  # history and the root; node 1 stays
        assert (got[33] == old[31 + 4]).all() and (got[34] == old[31 + 8]).all()
        assert (got[35:] == old[35:]).all()
    assert (pool[:, [2, 3, 5]] == before[:, [2, 3, 5]]).all()


# ---------------------------------------------------------------- host helpers of the library
@pytest.mark.parametrize("T", [1, 2, 7, 63, 64])
def test_tree_masks_match_the_definition(T):
    rng = np.random.default_rng(T)
    par = random_parents(rng, 5, T)
    lens = np.array([T, 0, 1, rng.integers(0, T + 1), T], np.int32)
    for ln in (None, lens):
        masks, depths = kvc.kv_tree_masks(par, ln)
        ref_m, ref_d = tree.tree_masks(par, ln)
        assert (masks.view(np.uint64) == ref_m).all() and (depths == ref_d).all()


def test_tree_masks_refuse_bad_trees():
    for par, lens, name in (([[-1, 1]], None, "INVALID"), ([[-1, -1]], None, "INVALID"), ([[-1, 0, 5]], None, "INVALID"),
                            ([[-1, 0]], [3], "INVALID"), ([[-1, 0]], [-1], "INVALID"), ([[0] * 65], None, "UNSUPPORTED")):
        with pytest.raises(kvc.KvcError) as e:
            kvc.kv_tree_masks(np.array(par, np.int32), lens)
        assert e.value.name == "KVC_ERR_" + name
    kvc.kv_tree_masks(np.array([[7, 0, 99]], np.int32), [2])  # the root's parent and entries behind a tree: not read
    assert kvc.kv_tree_masks(np.zeros((0, 4), np.int32))[0].shape == (0, 4)


def test_rope_turns_keep_far_angles():
    freq = 1e6 ** (-np.arange(0, 128, 2, dtype=np.float64) / 128)
    turns = kvc.kv_rope_turns(freq).view(np.uint64)
    for pos in (1, 4095, 131072, 2 ** 31 - 1):
        for f, t in zip(freq.tolist(), turns.tolist()):
            got = (pos * t % 2 ** 64) / 2 ** 64
            want = math.fmod(pos * f, 2 * math.pi) / (2 * math.pi)
            d = abs(got - want) % 1.0
            # a few roundings (2^-53) of the angle in turns on both sides, and the integer's own: half a unit of
            # 2^-64 turns per position
            assert min(d, 1 - d) < 6 * 2.0 ** -53 * (pos * f / (2 * math.pi) + 1) + pos * 2.0 ** -65, (pos, f)
    assert kvc.kv_rope_turns([0.0, 2 * math.pi]).view(np.uint64)[0] == 0
    for bad in ([-1.0], [float("nan")], [float("inf")]):
        with pytest.raises(kvc.KvcError):
            kvc.kv_rope_turns(bad)


# ---------------------------------------------------------------- refusals, before anything touches a device
P = ctypes.c_void_p(4096)  # a non-null, aligned address that no refused call follows
ODD = ctypes.c_void_p(4104)


def refused(fn, args, status, text=""):
    got = getattr(kvc._lib, fn)(*args)
    assert kvc.STATUS[got] == "KVC_ERR_" + status, (kvc.STATUS[got], kvc._lib.kvc_last_error_string())
    assert text in kvc._lib.kvc_last_error_string().decode()


def test_append_rope_refusals():
    base = dict(q=P, qs=256, k=P, ks=128, v=P, vs=128, n=2, Hq=4, Hkv=2, D=64, qw=None, kw=None, eps=1e-6, turns=P,
                rot=64, inter=0, pos=P, qo=ctypes.c_void_p(8192), ko=None, vo=None, kc=P, vc=P, NB=4, bs=16, slots=P,
                st=None)
    for change, status in ((dict(n=-1), "INVALID"), (dict(Hq=0), "INVALID"), (dict(D=96), "UNSUPPORTED"),
                           (dict(rot=24), "UNSUPPORTED"), (dict(rot=80), "UNSUPPORTED"), (dict(rot=-16), "UNSUPPORTED"),
                           (dict(inter=2), "INVALID"), (dict(bs=32), "UNSUPPORTED"), (dict(q=None), "INVALID"),
                           (dict(qo=None), "INVALID"), (dict(turns=None), "INVALID"), (dict(pos=None), "INVALID"),
                           (dict(slots=None), "INVALID"), (dict(kc=None), "INVALID"), (dict(NB=0), "INVALID"),
                           (dict(q=ODD), "INVALID"), (dict(kw=ODD), "INVALID"), (dict(vo=ODD), "INVALID"),
                           (dict(qs=250), "INVALID"), (dict(qs=248), "INVALID"), (dict(ks=64), "INVALID"),
                           (dict(qs=512, qo=P), "INVALID"), (dict(Hkv=70000), "UNSUPPORTED")):
        refused("kv_append_rope", list({**base, **change}.values()), status)
    assert kvc._lib.kv_append_rope(*{**base, "n": 0}.values()) == 0


def test_append_rope_refuses_outputs_that_overlap_its_rows():
    at = ctypes.c_void_p
    # two tokens of 4 + 2 + 2 heads of 64 in one projection: rows of 512 values (1024 bytes)
    base = dict(q=at(4096), qs=512, k=at(4096 + 512), ks=512, v=at(4096 + 768), vs=512, n=2, Hq=4, Hkv=2, D=64, qw=None,
                kw=None, eps=1e-6, turns=P, rot=64, inter=0, pos=P, qo=at(8192), ko=None, vo=None, kc=None, vc=None, NB=4,
                bs=16, slots=None, st=None)
    for change in (dict(qo=at(4096 + 512)), dict(qo=at(4096 - 1008)), dict(qo=at(4096 + 2032)), dict(ko=at(4096)),
                   dict(ko=at(4096 + 768)), dict(vo=at(4096 + 512)),
                   # packed rows: in place of one's own rows only, and not shifted
                   dict(ks=128, k=at(65536), ko=at(65536 + 16)), dict(ks=128, k=at(65536), vo=at(65536))):
        refused("kv_append_rope", list({**base, **change}.values()), "INVALID", "overlaps")


def test_tree_attention_refusals():
    base = dict(q=P, k=P, v=P, NB=64, table=P, mb=8, ctx=P, masks=P, lens=None, T=4, B=2, Hq=4, Hkv=2, D=64, bs=16,
                most=128, scale=0.125, out=P, od=0, ws=None, wb=0, st=None)
    for change, status in ((dict(T=0), "UNSUPPORTED"), (dict(T=65), "UNSUPPORTED"), (dict(Hq=5), "INVALID"),
                           (dict(Hq=130), "UNSUPPORTED"), (dict(D=80), "UNSUPPORTED"), (dict(bs=8), "UNSUPPORTED"),
                           (dict(masks=None), "INVALID"), (dict(ctx=None), "INVALID"), (dict(out=ODD), "INVALID"),
                           (dict(masks=ctypes.c_void_p(4100)), "INVALID"), (dict(most=129), "CAPACITY"),
                           (dict(od=2), "INVALID"), (dict(NB=0), "INVALID"), (dict(NB=2 ** 26), "UNSUPPORTED"),
                           (dict(scale=float("nan")), "INVALID"), (dict(B=-1), "INVALID"), (dict(B=70000), "UNSUPPORTED")):
        refused("paged_decode_tree_attention", list({**base, **change}.values()), status)
    assert kvc._lib.paged_decode_tree_attention(*{**base, "B": 0}.values()) == 0
    with pytest.raises(kvc.KvcError):
        kvc.paged_decode_tree_plan(1, 4, 2, 64, 100, 65)


def test_verify_refusals():
    base = dict(p=P, ps=100, q=P, qs=100, dt=1, tok=P, par=P, lens=None, u=P, B=2, T=4, V=100, distinct=0, path=P,
                plen=P, nxt=P, st=None)
    for change, status in ((dict(V=0), "INVALID"), (dict(T=0), "UNSUPPORTED"), (dict(T=65), "UNSUPPORTED"),
                           (dict(ps=99), "INVALID"), (dict(qs=99), "INVALID"), (dict(dt=2), "INVALID"),
                           (dict(distinct=2), "INVALID"), (dict(tok=None), "INVALID"), (dict(nxt=None), "INVALID"),
                           (dict(p=ctypes.c_void_p(4098)), "INVALID"), (dict(B=-1), "INVALID"),
                           (dict(V=2 ** 25, ps=2 ** 25, qs=2 ** 25), "UNSUPPORTED")):
        refused("draft_tree_verify", list({**base, **change}.values()), status)
    assert kvc._lib.draft_tree_verify(*{**base, "B": 0}.values()) == 0


def test_commit_refuses_new_lengths_among_its_inputs():
    hp = ctypes.c_void_p()
    cfg = kvc.KvcConfig(1, 4, 2, 64)._c()
    assert kvc._lib.kv_cache_create(ctypes.byref(cfg), P, P, ctypes.byref(hp)) == 0  # never followed below
    at = ctypes.c_void_p
    base = dict(h=hp, table=at(4096), mb=4, ctx=at(8192), lens=at(12288), path=at(16384), plen=at(20480), P=4, B=3,
                new=at(24576), st=None)
    try:
        for new in (4096, 4096 + 44, 8192, 8192 + 8, 8192 - 8, 12288, 16384 + 44, 20480, 20480 - 8):
            refused("kv_tree_commit", list({**base, "new": at(new)}.values()), "INVALID", "overlaps")
    finally:
        kvc.kv_cache_destroy(hp)


def test_commit_refusals():
    h = kvc.kv_cache_create(kvc.KvcConfig(1, 4, 2, 64))
    try:
        out = ctypes.c_void_p(8192)
        refused("kv_tree_commit", (None, P, 4, P, None, P, P, 4, 1, out, None), "INVALID", "null handle")
        refused("kv_tree_commit", (h, P, 4, P, None, P, P, 4, 1, out, None), "INVALID", "host-only")
    finally:
        kvc.kv_cache_destroy(h)
    hp = ctypes.c_void_p()
    cfg = kvc.KvcConfig(1, 4, 2, 64)._c()
    assert kvc._lib.kv_cache_create(ctypes.byref(cfg), P, P, ctypes.byref(hp)) == 0  # never followed below
    base = dict(h=hp, table=P, mb=4, ctx=P, lens=None, path=P, plen=P, P=4, B=1, new=ctypes.c_void_p(8192), st=None)
    try:
        for change, status in ((dict(P=0), "UNSUPPORTED"), (dict(P=65), "UNSUPPORTED"), (dict(new=P), "INVALID"),
                               (dict(path=None), "INVALID"), (dict(mb=0), "INVALID"), (dict(B=-1), "INVALID"),
                               (dict(B=70000), "UNSUPPORTED")):
            refused("kv_tree_commit", list({**base, **change}.values()), status)
        assert kvc._lib.kv_tree_commit(*{**base, "B": 0}.values()) == 0
    finally:
        kvc.kv_cache_destroy(hp)


# ---------------------------------------------------------------- the calls with their arguments as words
def test_calls_with_words_are_the_calls():
    words = lambda *a: struct.pack("=%dq" % len(a), *a)  # noqa: E731
    call = kvc._lib.kvc_call
    names = ("kv_append_rope", "paged_decode_tree_attention", "draft_tree_verify", "kv_tree_commit")
    for i, name in enumerate(names):
        n = len(getattr(kvc._lib, name).argtypes) - 1
        for which, w, count, text in ((i + 1, words(*[0] * (n + 1)), n + 1, f"{n} arguments"),
                                      (i + 1, words(*[0] * n), n - 1, f"{n} arguments"), (i + 1, None, n, "null pointer")):
            assert kvc.STATUS[call(which, w, count, None)] == "KVC_ERR_INVALID"
            assert text in kvc._lib.kvc_last_error_string().decode()
    for which in (0, 5, -1):
        assert kvc.STATUS[call(which, words(0), 1, None)] == "KVC_ERR_INVALID"
    # the commit's arguments in order: handle, table, max_blocks, lengths, tree lengths, path, its length, P, B, new
    assert kvc.STATUS[call(4, words(0, 4096, 4, 4096, 0, 4096, 4096, 4, 1, 8192), 10, None)] == "KVC_ERR_INVALID"
    assert "null handle" in kvc._lib.kvc_last_error_string().decode()
    assert kvc.STATUS[call(4, words(0, 4096, 4, 4096, 0, 4096, 4096, 2 ** 32 + 4, 1, 8192), 10, None)] == "KVC_ERR_INVALID"
    assert "beyond its type" in kvc._lib.kvc_last_error_string().decode()
    # a float is a double: the tree's scale, place 16
    args = [4096, 4096, 4096, 64, 4096, 8, 4096, 4096, 0, 4, 2, 4, 2, 64, 16, 128, float("nan"), 4096, 0, 0, 0]
    w = struct.pack("=16qd4q", *args)
    assert kvc.STATUS[call(2, w, 21, None)] == "KVC_ERR_INVALID"
    assert "scale" in kvc._lib.kvc_last_error_string().decode()
    with pytest.raises(kvc.KvcError, match="unknown call"):
        kvc.kvc_call(9, words(0))
    with pytest.raises(ValueError):
        kvc.kvc_call(1, b"1234567")


def test_the_steps_kernels_read_nothing_as_constant():
    """They are launched before the kernel in front of them has ended, and may read what it writes: no load through the
    read-only path, which is defined only for data that is constant for a kernel's whole life, and no pointer that is
    promised to be read alone."""
    csrc = os.path.join(os.path.dirname(kvc.__file__), "csrc")
    for name in ("append_rope.cu", "tree_attention.cu", "tree_verify.cu", "tree_commit.cu"):
        with open(os.path.join(csrc, name)) as f:
            code = re.sub(r"//.*", "", f.read())
        assert not re.search(r"__ldg|__restrict__|\.nc\b|ld_nc", code), name


# ---------------------------------------------------------------- outputs among the inputs, or among each other
def at(i, off=0):
    """The i-th of addresses 16 MB apart, more than any buffer below holds."""
    return ctypes.c_void_p((i << 24) + off)


def test_append_rope_refuses_outputs_among_all_it_reads():
    base = dict(q=at(1), qs=256, k=at(2), ks=128, v=at(3), vs=128, n=20, Hq=4, Hkv=2, D=64, qw=at(4), kw=at(5), eps=1e-6,
                turns=at(6), rot=64, inter=0, pos=at(7), qo=at(8), ko=at(9), vo=at(10), kc=at(11), vc=at(12), NB=4, bs=16,
                slots=at(13), st=None)
    cache = 4 * 2 * 16 * 64 * 2
    for change in (dict(kc=at(1)), dict(vc=at(2, -16)), dict(kc=at(3, 20 * 256 - 16)), dict(kc=at(1, 16 - cache)),
                   dict(qo=at(4)), dict(ko=at(5, 112)), dict(vo=at(6, 240)), dict(qo=at(7, 64)), dict(qo=at(13, 144)),
                   dict(kc=at(4)), dict(vc=at(13)), dict(kc=at(7, 64)), dict(ko=at(8)), dict(vo=at(9, 16)),
                   dict(qo=at(11, 16)), dict(vo=at(12)), dict(vc=at(11, cache - 16)), dict(qs=2 ** 60, qo=at(1, 2 ** 40))):
        refused("kv_append_rope", list({**base, **change}.values()), "INVALID", "overlaps")


def test_tree_attention_refuses_an_output_among_its_inputs():
    base = dict(q=at(1), k=at(2), v=at(3), NB=64, table=at(4), mb=8, ctx=at(5), masks=at(6), lens=at(7), T=4, B=2, Hq=4,
                Hkv=2, D=64, bs=16, most=128, scale=0.125, out=at(8), od=0, ws=None, wb=0, st=None)
    size = 2 * 4 * 4 * 64
    for change in (dict(out=at(1)), dict(out=at(1, size * 2 - 16)), dict(out=at(1, 16 - size * 2)),
                   dict(out=at(1, 16 - size * 4), od=1), dict(out=at(2)), dict(out=at(3, 64 * 2 * 16 * 64 * 2 - 16)),
                   dict(out=at(4, 48)), dict(out=at(5)), dict(out=at(6, 48)), dict(out=at(7))):
        refused("paged_decode_tree_attention", list({**base, **change}.values()), "INVALID", "overlaps")


def test_verify_refuses_outputs_among_its_inputs_and_each_other():
    base = dict(p=at(1), ps=104, q=at(2), qs=100, dt=1, tok=at(3), par=at(4), lens=at(5), u=at(6), B=3, T=4, V=100,
                distinct=0, path=at(7), plen=at(8), nxt=at(9), st=None)
    for change in (dict(path=at(3)), dict(path=at(4, 44)), dict(plen=at(5)), dict(nxt=at(5, 8)), dict(plen=at(6, 44)),
                   dict(nxt=at(3, 8)), dict(path=at(1, 11 * 104 * 4 + 396)), dict(path=at(2, -44)),
                   dict(nxt=at(1, 8), dt=0), dict(plen=at(7, 44)), dict(nxt=at(8, 8)), dict(path=at(9, -44))):
        refused("draft_tree_verify", list({**base, **change}.values()), "INVALID", "overlaps")


def test_commit_refuses_lengths_and_tables_in_its_pools():
    hp = ctypes.c_void_p()
    cfg = kvc.KvcConfig(2, 4, 2, 64)._c()
    assert kvc._lib.kv_cache_create(ctypes.byref(cfg), at(1), at(2), ctypes.byref(hp)) == 0  # never followed below
    size = 2 * 4 * 2 * 16 * 64 * 2
    base = dict(h=hp, table=at(3), mb=4, ctx=at(4), lens=at(5), path=at(6), plen=at(7), P=4, B=3, new=at(8), st=None)
    try:
        for change in (dict(new=at(1)), dict(new=at(2, size - 4)), dict(table=at(1, size - 4)), dict(ctx=at(2, -8)),
                       dict(path=at(1, 64)), dict(plen=at(2)), dict(lens=at(1))):
            refused("kv_tree_commit", list({**base, **change}.values()), "INVALID", "overlaps")
    finally:
        kvc.kv_cache_destroy(hp)


def test_tree_masks_refuse_outputs_among_their_inputs():
    par, masks = np.zeros((2, 4), np.int32), np.zeros((2, 4), np.int64)
    p = lambda a, off=0: ctypes.c_void_p(a.ctypes.data + off)  # noqa: E731
    for args in ((p(masks, 32), None, 2, 4, p(masks), None), (p(par), None, 2, 4, p(masks), p(par)),
                 (p(par), p(masks, 56), 2, 4, p(masks), None), (p(par), None, 2, 4, p(masks), p(masks, 32))):
        refused("kv_tree_masks", args, "INVALID", "overlaps")


def test_arrays_that_are_not_aligned_to_their_types_are_refused():
    """A misaligned load would be a fault on the device."""
    rope = dict(q=at(1), qs=256, k=at(2), ks=128, v=at(3), vs=128, n=20, Hq=4, Hkv=2, D=64, qw=None, kw=None, eps=1e-6,
                turns=at(6), rot=64, inter=0, pos=at(7), qo=at(8), ko=None, vo=None, kc=at(11), vc=at(12), NB=4, bs=16,
                slots=at(13), st=None)
    attention = dict(q=at(1), k=at(2), v=at(3), NB=64, table=at(4), mb=8, ctx=at(5), masks=at(6), lens=at(7), T=4, B=2,
                     Hq=4, Hkv=2, D=64, bs=16, most=128, scale=0.125, out=at(8), od=0, ws=None, wb=0, st=None)
    verify = dict(p=at(1), ps=104, q=at(2), qs=100, dt=1, tok=at(3), par=at(4), lens=at(5), u=at(6), B=3, T=4, V=100,
                  distinct=0, path=at(7), plen=at(8), nxt=at(9), st=None)
    hp = ctypes.c_void_p()
    cfg = kvc.KvcConfig(2, 4, 2, 64)._c()
    assert kvc._lib.kv_cache_create(ctypes.byref(cfg), at(1), at(2), ctypes.byref(hp)) == 0  # never followed below
    commit = dict(h=hp, table=at(3), mb=4, ctx=at(4), lens=at(5), path=at(6), plen=at(7), P=4, B=3, new=at(8), st=None)
    try:
        for fn, base, arrays in (("kv_append_rope", rope, dict(turns=4, pos=2, slots=4)),
                                 ("paged_decode_tree_attention", attention, dict(table=2, ctx=1, masks=4, lens=2)),
                                 ("draft_tree_verify", verify, dict(p=2, q=1, tok=2, par=3, lens=2, u=2, path=1, plen=2, nxt=2)),
                                 ("kv_tree_commit", commit, dict(table=2, ctx=1, lens=2, path=3, plen=2, new=2))):
            for name, off in arrays.items():
                refused(fn, list({**base, name: ctypes.c_void_p(base[name].value + off)}.values()), "INVALID", "aligned")
    finally:
        kvc.kv_cache_destroy(hp)


def test_contexts_beyond_32_bit_positions_are_refused():
    """The plan's number of key tiles overflowed for the last 127 lengths below 2^31: a workspace of nothing."""
    base = dict(q=at(1), k=at(2), v=at(3), NB=64, table=at(4), mb=2 ** 27, ctx=at(5), masks=at(6), lens=None, T=4, B=1,
                Hq=4, Hkv=2, D=64, bs=16, most=2 ** 30 + 1, scale=0.125, out=at(8), od=0, ws=None, wb=0, st=None)
    for most in (2 ** 30 + 1, 2 ** 31 - 1):
        refused("paged_decode_tree_attention", list({**base, "most": most}.values()), "UNSUPPORTED", "max_context_len")
        with pytest.raises(kvc.KvcError) as e:
            kvc.paged_decode_tree_plan(1, 4, 2, 64, most, 4)
        assert e.value.name == "KVC_ERR_UNSUPPORTED"


def test_append_rope_refuses_an_eps_that_no_norm_has():
    base = dict(q=at(1), qs=256, k=at(2), ks=128, v=at(3), vs=128, n=20, Hq=4, Hkv=2, D=64, qw=None, kw=at(5), eps=1e-6,
                turns=None, rot=0, inter=0, pos=None, qo=at(8), ko=at(9), vo=None, kc=None, vc=None, NB=0, bs=16, slots=None,
                st=None)
    for eps in (-1e-6, float("nan"), float("inf")):
        refused("kv_append_rope", list({**base, "eps": eps}.values()), "INVALID", "eps")


def test_host_tensors_are_refused_as_such():
    """Also where there is no GPU, whose current device cannot be asked for."""
    t = lambda dt, *shape: torch.zeros(shape, dtype=dt)  # noqa: E731
    f16, f32, i32, i64 = torch.float16, torch.float32, torch.int32, torch.int64
    h = kvc.kv_cache_create(kvc.KvcConfig(1, 4, 2, 64))
    try:
        for call in (lambda: kvc.kv_append_rope(t(f16, 3, 4, 64), t(f16, 3, 2, 64), t(f16, 3, 2, 64), None, None,
                                                t(f16, 3, 4, 64)),
                     lambda: kvc.paged_decode_tree_attention(t(f16, 1, 2, 4, 64), t(f16, 4, 2, 16, 64),
                                                             t(f16, 4, 2, 16, 64), t(i32, 1, 4), t(i32, 1), t(i64, 1, 2),
                                                             0.125, t(f16, 1, 2, 4, 64), None, 64),
                     lambda: kvc.draft_tree_verify(t(f32, 1, 2, 9), t(f32, 1, 2, 9), t(i32, 1, 2), t(i32, 1, 2),
                                                   t(f32, 1, 2), t(i32, 1, 2), t(i32, 1), t(i32, 1)),
                     lambda: kvc.kv_tree_commit(h, t(i32, 1, 4), t(i32, 1), t(i32, 1, 4), t(i32, 1), t(i32, 1))):
            with pytest.raises(ValueError, match="must be on a CUDA device"):
                call()
    finally:
        kvc.kv_cache_destroy(h)


def test_commit_refuses_a_destroyed_cache():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    args = (i32(1, 4), i32(1), i32(1, 4), i32(1), i32(1))
    h = kvc.kv_cache_create(kvc.KvcConfig(1, 4, 2, 64))
    with pytest.raises(ValueError, match="CUDA"):  # open: it is the tensors that are refused
        kvc.kv_tree_commit(h, *args)
    kvc.kv_cache_destroy(h)
    for handle in (h, 0, None):
        for prepare in (False, True):
            with pytest.raises(ValueError, match="not an open cache"):
                kvc.kv_tree_commit(handle, *args, prepare=prepare)
