"""Numerics of a tree-drafted step where scores, weights and angles are far apart, against the definitions in fp64.

Every output of the tree attention is held to its own row's bound, with e_i the relative error of key i's weight w_i:
  |err| <= sum_i w_i e_i (|v_i| + |out|) + 2^-36 max(w) sum_i (|v_i| + |out|) + sums + the store's half step,
  e_i = the weight's own rounding (2^-11 with fp16 outputs, 2^-22 with fp32 ones) + its exponential (2^-22)
        + D 2^-24 of the score's terms' magnitudes + 4 * 2^-24 of its exponent (its distance to the row's largest
        score, and the 11 ln 2 < 8 by which weights are carried higher) + 2^-18 for the rescalings of a row's state
        (at most 16 factors of 2^-22),
  sums = 2^-23 per product instruction of 16 keys of numerator and row sum, and 2^-21 inside one.
The second term is what the call documents for weights below fp16's normal range.
"""
import numpy as np
import pytest
import torch

import workloads
from test_gpu_tree import MANY, TREES, Tree, dev, host, kvc, many  # noqa: F401  (kvc is a fixture)
from oracle import tree

pytestmark = pytest.mark.gpu


def rows_and_bounds(w, out_dtype, b, hk, tiles=False):
    """For the rows (node, query head of KV head hk) of sequence b: fp64 outputs and their bounds [rows][D]; with tiles
    also the outputs [tile][rows][D] that come of leaving out a tile of 128 keys."""
    G, L, n, D = w.Hq // w.Hkv, int(w.lens[b]), int(w.ctx[b]), w.D
    half = out_dtype == torch.float16
    hist = n - L
    K, V = (tree.rows_of(c[:, hk:hk + 1], w.table[b], n)[:, 0].astype(np.float64) for c in (w.k, w.v))
    q = w.q[b, :L, hk * G:(hk + 1) * G].astype(np.float64).reshape(L * G, D)
    seen = np.ones((L, n), bool)
    seen[:, hist:] = (w.masks[b, :L, None] >> np.arange(L, dtype=np.uint64)) & np.uint64(1) == 1
    seen = np.repeat(seen, G, 0)
    x = np.where(seen, q @ np.where(np.isfinite(K), K, 0).T * w.scale, -np.inf)
    top = x.max(1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(x - top)
    total = np.maximum(e.sum(1, keepdims=True), 1e-300)
    p = e / total
    out = p @ V
    far = np.where(seen, top - x, 0.0)
    terms = np.abs(q) @ np.abs(K).T * abs(w.scale)
    rel = (2.0 ** -11 if half else 2.0 ** -22) + 2.0 ** -22 + D * 2.0 ** -24 * terms + 4 * 2.0 ** -24 * (far + 8) + 2.0 ** -18
    A, size = np.abs(V), np.abs(out)
    pr = p * rel
    bound = pr @ A + pr.sum(1, keepdims=True) * size
    bound += 2.0 ** -36 / total * (seen @ A + seen.sum(1, keepdims=True) * size)
    bound += (n / 16 * 2.0 ** -23 + 2.0 ** -21) * (p @ A + size)
    bound = 1.01 * bound + ((2.0 ** -11 if half else 2.0 ** -24) * size + 2.0 ** -25)
    if not tiles:
        return out, bound
    starts = np.arange(0, n, 128)
    part = np.stack([e[:, s:s + 128] @ V[s:s + 128] for s in starts])
    mass = np.add.reduceat(e, starts, 1).T[:, :, None]
    with np.errstate(invalid="ignore", divide="ignore"):
        without = (out * total - part) / (total - mass)
    return out, bound, without


def check(w, got, out_dtype, what, rows=None):
    G = w.Hq // w.Hkv
    for b in range(len(w.ctx)):
        L = int(w.lens[b])
        assert (got[b, L:] == 55.0).all(), f"{what}: a row behind a tree was written"
        for hk in range(w.Hkv if L else 0):
            ref, bound = rows_and_bounds(w, out_dtype, b, hk)
            have = got[b, :L, hk * G:(hk + 1) * G].reshape(L * G, w.D)
            err = np.abs(have - ref)
            assert (err <= bound).all(), (f"{what}, sequence {b}, KV head {hk}: {np.nanmax(err / bound):.3f} of the "
                                          f"bound, {int((~(err <= bound)).sum())} outputs")


# ---------------------------------------------------------------- scores far from zero
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("D,Hq,Hkv,hist,T", [(64, 2, 1, 0, 1), (128, 8, 2, 700, 9), (64, 14, 2, 3000, 40),
                                             (128, 1, 1, 20000, 3)])
def test_scores_beyond_what_fp32_resolves(kvc, D, Hq, Hkv, hist, T, out_dtype):
    """Finite fp16 rows whose scores reach 2^38: the softmax takes the largest one alone, wherever it stands, and keys
    of equal scores share it."""
    w = Tree(60 + D + T, [hist], [T], T, Hq, Hkv, D)
    rng = np.random.default_rng([61, D, T])
    n = hist + T
    w.q[:] = 60000
    pos = np.arange(n)
    key = np.full((n, Hkv), 20000, np.float16)
    best = rng.integers(0, hist + 1, Hkv)  # node 0, the last choice, is seen by its own row alone below
    w.masks[:] = np.uint64(1) << np.arange(T, dtype=np.uint64)
    for h in range(Hkv):
        key[rng.permutation(n)[:n // 2], h] = 40000
        key[hist:, h] = 20000
        key[best[h], h] = 60000
        w.k[w.table[0][pos // 16], h, pos % 16] = key[:, h, None]
    for sign in (1, -1):
        w.scale = sign * D ** -0.5
        if sign < 0:
            w.q[:] = -60000
        got = w.run(kvc, out_dtype)
        assert np.isfinite(got).all()
        V = tree.rows_of(w.v, w.table[0], n).astype(np.float64)
        for t in range(T):
            for h in range(Hq):
                hk = h // (Hq // Hkv)
                sees = key[:, hk].astype(np.float64)
                sees[hist:][np.arange(T) != t] = 0
                win = sees == sees.max()
                want = V[win, hk].mean(0)
                few = (win.sum() / 16 * 2.0 ** -23 + 2.0 ** -20) * np.abs(V[win, hk]).mean(0)
                tol = few + 2.0 ** -25 + (2.0 ** -11 if out_dtype == torch.float16 else 2.0 ** -24) * np.abs(want)
                assert (np.abs(got[0, t, h] - want) <= tol).all(), (sign, t, h)


# ---------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("nats", [9.0, 16.0, 17.4, 20.0])
@pytest.mark.parametrize("D,Hq,Hkv,T,at", [(64, 2, 1, 3, 0), (128, 8, 1, 20, 0), (64, 2, 2, 2, 65535),
                                           (128, 4, 2, 64, 40000)])
def test_a_long_tail_below_one_key(kvc, D, Hq, Hkv, T, at, nats, out_dtype):
    """An attention sink: one key of 65,536 with a value of 0, `nats` above all others, whose values are about 1.  What
    comes out is the others' mass, whatever part of the context the sink stands in."""
    hist = 65536
    w = Tree(62, [hist], [T], T, Hq, Hkv, D)
    n = hist + T
    w.scale = 1.0
    w.q[:] = 0
    w.q[..., 0] = 8.0
    pos = np.arange(n)
    w.k[w.table[0][pos // 16], :, pos % 16] = 0
    w.k[w.table[0][at // 16], :, at % 16, 0] = nats / 8
    v = np.abs(w.v) * np.float16(0.25) + np.float16(1)
    w.v[w.table[0][pos // 16], :, pos % 16] = v[w.table[0][pos // 16], :, pos % 16]
    w.v[w.table[0][at // 16], :, at % 16] = 0
    got = w.run(kvc, out_dtype)
    mass = n * np.exp(-nats)
    assert (np.abs(got[0] / (mass / (1 + mass)) - 1.2) < 0.2).all()
    check(w, got, out_dtype, f"sink {nats} nats above")


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
def test_weights_of_every_size(kvc, out_dtype):
    """Scores spread over 30 nats, their largest anywhere, so that every range of weights carries some of the output."""
    w = Tree(63, [40000, 7000], [10, 3], 10, 8, 2, 64, sharp=6.0)
    w.v[:] = np.where(np.isnan(w.v), w.v, np.abs(w.v))
    check(w, w.run(kvc, out_dtype), out_dtype, "sharp scores")


# ---------------------------------------------------------------- each row by its own bound
LONG = [i for i, t in enumerate(TREES) if max(t[0]) >= 500] + [5, 6, 13]


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("case", LONG)
def test_every_output_within_its_rows_bound(kvc, case, out_dtype):
    hist, lens, T, Hq, Hkv, D, empty = TREES[case]
    w = Tree(70 + case, hist, lens, T, Hq, Hkv, D, empty)
    check(w, w.run(kvc, out_dtype), out_dtype, f"case {case}")


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("case", [2, 4, 6])
def test_every_output_of_many_sequences_within_its_rows_bound(kvc, case, out_dtype):
    B, T, Hq, Hkv, D, far, none = MANY[case]
    w = many(case, T, Hq, Hkv, D, B, far, none)
    check(w, w.run(kvc, out_dtype), out_dtype, f"many, case {case}")


PLANTED = [
    # hist, tree lens, T, Hq, Hkv, D: one cluster of several CTAs; several clusters; one, two and four pairs of row tiles
    ([4000, 2100], [12, 12], 12, 8, 1, 128),
    ([30000, 9000, 700], [5, 5, 5], 5, 2, 1, 64),
    ([20000], [40], 40, 8, 1, 128),
    ([9000], [64], 64, 14, 2, 64),
    ([6000, 200], [64, 64], 64, 16, 1, 64),
    ([65536], [16], 16, 4, 1, 128),
]


@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("case", range(len(PLANTED)))
def test_no_tile_of_keys_is_lost(kvc, case, out_dtype):
    """Every tile of 128 keys of the history holds a key that carries much of some row's mass: an output without any one
    of them lies far outside the bound, which is shown on the definition first."""
    hist, lens, T, Hq, Hkv, D = PLANTED[case]
    w = Tree(80 + case, hist, lens, T, Hq, Hkv, D)
    rng = np.random.default_rng([81, case])
    G = Hq // Hkv
    for b, h in enumerate(hist):
        for hk in range(Hkv):
            for i, s in enumerate(range(0, h, 128)):
                t, g = divmod(i % (lens[b] * G), G)
                row = w.q[b, t, hk * G + g].astype(np.float64)
                at = s + int(rng.integers(0, min(128, h - s)))
                w.k[w.table[b][at // 16], hk, at % 16] = row * (np.log(h) / (w.scale * (row @ row)))
    got = w.run(kvc, out_dtype)
    check(w, got, out_dtype, f"planted case {case}")
    for b, h in enumerate(hist):
        for hk in range(Hkv):
            ref, bound, without = rows_and_bounds(w, out_dtype, b, hk, tiles=True)
            whole = h // 128  # (the tile that reaches into the tree may be all that a row of it sees)
            lost = np.abs(without[:whole] - ref) > 3 * bound
            assert lost.any((1, 2)).all(), f"case {case}: leaving out tiles {np.flatnonzero(~lost.any((1, 2)))} would pass"


# ---------------------------------------------------------------- norm, rotation, append
@pytest.mark.parametrize("D,rot,inter", [(64, 32, False), (64, 16, True), (128, 64, True), (128, 96, False), (64, 0, False)])
def test_an_infinity_behind_the_rotated_values_stays_there(kvc, D, rot, inter):
    """A row with an infinity is normed to NaN where that is and to 0 elsewhere; values behind rot_dim take nothing from
    one another."""
    n, H = 5, 3
    rng = np.random.default_rng([90, D, rot])
    x = workloads.normal_f16(rng, (n, H, D))
    at = rng.integers(rot, D, n)
    x[np.arange(n), 1, at] = np.inf
    x[0, 1, at[0]] = -np.inf
    w = workloads.normal_f16(rng, (D,))
    pos = np.arange(n, dtype=np.int32) + 3
    freq = 1e4 ** (-np.arange(0, rot, 2) / max(rot, 1))
    out, k_out = (torch.empty((n, H, D), dtype=torch.float16, device="cuda") for _ in range(2))
    q = dev(x)
    kvc.kv_append_rope(q, q, q, dev(pos), dev(kvc.kv_rope_turns(freq)), out, q_weight=dev(w), k_weight=dev(w),
                       interleaved=inter, k_out=k_out)
    with np.errstate(invalid="ignore"):
        ref = tree.norm_rotate(x, w, 1e-6, pos[:, None] * freq, inter)
    hit = np.zeros((n, D), bool)
    hit[np.arange(n), at] = True
    assert (np.isnan(ref[:, 1]) == hit).all() and (ref[:, 1][~hit] == 0).all()
    for got in (host(out), host(k_out)):
        assert (np.isnan(got) == np.isnan(ref)).all() and (got[:, 1][~hit] == 0).all()
        rest = [0, 2]  # heads without one
        assert (np.abs(got[:, rest] - ref[:, rest]) <= 2.0 ** -10 * np.abs(ref[:, rest]) + 2.0 ** -14).all()


@pytest.mark.parametrize("pos", [1, 3, 2 ** 16 + 1, 2 ** 31 - 1, -1])
def test_angles_are_rounded_to_the_nearest(kvc, pos):
    """An angle is within 2^-33 turn (the product rounded to 2^-32) and half an fp32 step (2^-24 of at most half a
    turn) of position x frequency; here it is that of (0, 65504) turned by about 2^-32 turn."""
    D = 64
    far = [2 ** 32 - 1 - 5 * i if i % 2 else 2 ** 31 + 1 + 5 * i for i in range(D // 2)]  # position x frequency
    turns = np.array([x * pow(pos % 2 ** 64, -1, 2 ** 64) % 2 ** 64 for x in far], np.uint64)
    q = np.zeros((1, 1, D), np.float16)
    q[..., D // 2:] = 65504
    out = torch.empty((1, 1, D), dtype=torch.float16, device="cuda")
    d = dev(q)
    kvc.kv_append_rope(d, d, d, dev(np.array([pos], np.int32)), dev(turns.view(np.int64)), out)
    angle = np.array(far, np.float64) * (2 * np.pi / 2.0 ** 64)
    half = np.abs(angle) * 2.0 ** -24 + 2 * np.pi * 2.0 ** -33
    got = host(out)[0, 0].astype(np.float64)
    for have, want in ((got[:D // 2], -65504 * np.sin(angle)), (got[D // 2:], 65504 * np.cos(angle))):
        # cosine, sine, product: 2^-22; the angle's error turns the vector; the store
        bound = 65504 * half + 2.0 ** -22 * np.abs(want) + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
        assert (np.abs(have - want) <= bound).all(), np.max(np.abs(have - want) / bound)
