"""Numerics of a tree-drafted step where scores, weights and angles are far apart, against the definitions in fp64.
"""
import numpy as np
import pytest
import torch

from test_gpu_tree import Tree, kvc  # noqa: F401  (kvc is a fixture)
from oracle import tree

pytestmark = pytest.mark.gpu


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
