"""Tree-drafted decoding on the GPU against the fp64 definitions (oracle/tree.py).

Tolerances count the roundings a path makes: fp16 stores round by 2^-11 of a value (2^-25 among subnormals), fp32
sums of N terms by N 2^-24 of the terms' magnitudes, softmax weights as the call documents.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import tree
from parity import F16_NAN_BITS

pytestmark = pytest.mark.gpu


@pytest.fixture
def kvc():
    import paged_kv_cache_27_gb300 as m
    m.kvc_device_error_flags(clear=True)
    yield m
    m.kvc_set_checked_mode(False)
    m.kvc_device_error_flags(clear=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().cpu().numpy()


# ---------------------------------------------------------------- norm, rotation, append
def check_rows(got, raw, weight, eps, angle, inter, what):
    """fp16 rows got [n][H][D] against the definition on raw rows."""
    ref = tree.norm_rotate(raw, weight, eps, angle, inter)
    # fp32 steps in front of the store: the sum of squares (D terms, halved by the root), root, two products, two
    # rotation products and a sum, cosine and sine: below 2^-24 (D / 2 + 16) of the pair's magnitude; the angle's own
    # 2^-25 turns is 2^-22.3 radians
    mag = np.abs(tree.norm_rotate(raw, weight, eps, np.zeros((len(raw), 0)), inter))
    pairs = angle.shape[1]
    pair_mag = mag.copy()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + pairs)
        pair_mag[..., a] = pair_mag[..., b] = mag[..., a] + mag[..., b]
    D = raw.shape[-1]
    bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + ((D / 2 + 16) * 2.0 ** -24 + 2.0 ** -22) * pair_mag
    err = np.abs(got.astype(np.float64) - ref)
    assert (err <= bound).all(), f"{what}: {np.max(err / bound):.3f} of the bound"


APPEND = [
    # n, Hq, Hkv, D, rot, interleaved, q norm, k norm, first position
    (1, 14, 2, 64, 64, False, True, True, 0),
    (1, 1, 1, 64, 64, True, True, True, 2 ** 31 - 2),
    (7, 32, 8, 128, 128, False, True, True, 131072),
    (33, 14, 2, 64, 32, True, False, False, 100),
    (130, 8, 8, 128, 64, False, True, False, 17),
    (5, 3, 1, 64, 16, False, False, True, -5),
    (2500, 14, 2, 64, 48, False, True, True, 1000),
    (700, 5, 1, 128, 0, False, True, True, 0),
    (300, 64, 1, 64, 64, True, True, True, 7),
    (9, 2, 2, 128, 112, True, True, True, 50000),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_rope(kvc, case):
    n, Hq, Hkv, D, rot, inter, qn, kn, pos0 = APPEND[case]
    rng = np.random.default_rng([50, case])
    qkv = workloads.normal_f16(rng, (n, (Hq + 2 * Hkv) * D + 8 * (case % 3)))
    qkv[0, :D] *= 100
    d = dev(qkv)
    q, k, v = (d[:, a * D:b * D].unflatten(1, (-1, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    qw, kw = (workloads.normal_f16(rng, (D,)) for _ in range(2))
    freq = 1e4 ** (-np.arange(0, rot, 2, dtype=np.float64) / max(rot, 1))
    pos = (pos0 + np.arange(n) % 2).astype(np.int32)
    NB = n // 16 + 3
    slots = rng.permutation(NB * 16)[:n].astype(np.int64)
    if n > 4:
        slots[3] = -1
    kc, vc = (torch.full((NB, Hkv, 16, D), F16_NAN_BITS, dtype=torch.int16, device="cuda").view(torch.float16)
              for _ in range(2))
    q_out = torch.empty((n, Hq, D), dtype=torch.float16, device="cuda")
    k_out, v_out = (torch.empty((n, Hkv, D), dtype=torch.float16, device="cuda") for _ in range(2))
    kvc.kvc_set_checked_mode(case % 2 == 1)
    kvc.kv_append_rope(q, k, v, dev(pos) if rot else None, dev(kvc.kv_rope_turns(freq)) if rot else None, q_out, kc, vc,
                       dev(slots), q_weight=dev(qw) if qn else None, k_weight=dev(kw) if kn else None, eps=1e-5,
                       interleaved=inter, k_out=k_out, v_out=v_out)
    assert kvc.kvc_device_error_flags() == 0
    angle = pos[:, None].astype(np.float64) * freq
    check_rows(host(q_out), host(q), qw if qn else None, 1e-5, angle, inter, "q")
    check_rows(host(k_out), host(k), kw if kn else None, 1e-5, angle, inter, "k")
    assert (host(v_out).view(np.uint16) == host(v.contiguous()).view(np.uint16)).all()
    if not qn and not rot:
        assert (host(q_out).view(np.uint16) == host(q.contiguous()).view(np.uint16)).all()
    for cache, rows in ((kc, k_out), (vc, v_out)):
        want = np.full((NB * 16, Hkv, D), F16_NAN_BITS, np.uint16)
        keep = slots >= 0
        want[slots[keep]] = host(rows).view(np.uint16)[keep]
        got = host(cache).view(np.uint16).transpose(0, 2, 1, 3).reshape(NB * 16, Hkv, D)
        assert (got == want).all()


def test_append_rope_in_place_and_without_a_cache(kvc):
    rng = np.random.default_rng(51)
    n, Hq, Hkv, D = 40, 14, 2, 64
    q, k, v = (dev(workloads.normal_f16(rng, (n, H, D))) for H in (Hq, Hkv, Hkv))
    turns, pos = dev(kvc.kv_rope_turns(1e4 ** (-np.arange(0, D, 2) / D))), dev(np.arange(n, dtype=np.int32))
    a, b = torch.empty_like(q), torch.empty_like(k)
    kvc.kv_append_rope(q, k, v, pos, turns, a, k_out=b)
    kvc.kv_append_rope(q, k, v, pos, turns, q, k_out=k, v_out=v)
    assert torch.equal(q, a) and torch.equal(k, b)
    # no tokens; a bad slot is flagged and skipped
    kvc.kv_append_rope(q[:0], k[:0], v[:0], pos[:0], turns, q[:0])
    kc = torch.zeros((4, Hkv, 16, D), dtype=torch.float16, device="cuda")
    slots = torch.full((n,), 64, dtype=torch.int64, device="cuda")
    slots[1] = 63
    kvc.kv_append_rope(q, k, v, pos, turns, a, kc, kc.clone(), slots)
    assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["SLOT"]
    assert int((kc != 0).any(-1).sum()) == Hkv
    kvc.kvc_set_checked_mode(True)
    with pytest.raises(kvc.KvcError) as e:
        kvc.kv_append_rope(q, k, v, pos, turns, a, kc, kc.clone(), slots)
    assert e.value.name == "KVC_ERR_CAPACITY"


@pytest.mark.parametrize("n,Hq,Hkv,D", [(6000, 32, 8, 128), (12000, 32, 8, 64)])
def test_append_rope_of_a_long_prompt_is_its_parts(kvc, n, Hq, Hkv, D):
    """More rows than L2 holds go another way through it; the rows are the same."""
    g = torch.Generator(device="cuda").manual_seed(n)
    qkv = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g, device="cuda", dtype=torch.float16)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split((Hq * D, Hkv * D, Hkv * D), 1))
    w = torch.rand(2, D, generator=g, device="cuda").half()
    turns, pos = dev(kvc.kv_rope_turns(1e4 ** (-np.arange(0, D, 2) / D))), torch.arange(n, dtype=torch.int32, device="cuda")
    slots = torch.randperm(n, generator=g, device="cuda")
    got = []
    for step in (n, 500):
        out = torch.zeros((n, Hq, D), dtype=torch.float16, device="cuda")
        kc, vc = (torch.zeros((-(-n // 16), Hkv, 16, D), dtype=torch.float16, device="cuda") for _ in range(2))
        for a in range(0, n, step):
            s = slice(a, a + step)
            kvc.kv_append_rope(q[s], k[s], v[s], pos[s], turns, out[s], kc, vc, slots[s], q_weight=w[0], k_weight=w[1])
        got.append((out, kc, vc))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    check_rows(host(got[0][0][-3:]), host(q[-3:]), host(w[0]), 1e-6,
               np.arange(n - 3, n)[:, None] * (1e4 ** (-np.arange(0, D, 2) / D)), False, "last rows")


# ---------------------------------------------------------------- tree attention
class Tree:
    """Random queries, caches and masks; everything past a context, and every block no sequence owns, is NaN."""

    def __init__(self, seed, hist, lens, T, Hq, Hkv, D, empty_rows=False, sharp=1.0):
        rng = np.random.default_rng([52, seed])
        self.T, self.Hq, self.Hkv, self.D, B = T, Hq, Hkv, D, len(hist)
        self.lens = np.array(lens, np.int32)
        self.ctx = (np.array(hist) + self.lens).astype(np.int32)
        nblk = [-(-int(c) // 16) for c in self.ctx]
        NB = sum(nblk) + 2
        perm = rng.permutation(NB).astype(np.int32)
        self.table = np.full((B, max(max(nblk), 1)), -7, np.int32)  # entries behind a context are not read
        at = 0
        for b, n in enumerate(nblk):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.q = (workloads.normal_f16(rng, (B, T, Hq, D)) * np.float16(sharp)).astype(np.float16)
        self.k, self.v = (workloads.normal_f16(rng, (NB, Hkv, 16, D)) for _ in range(2))
        owned = np.zeros((NB, 16), bool)
        for b, c in enumerate(self.ctx):
            p = np.arange(c)
            owned[self.table[b][p // 16], p % 16] = True
        for x in (self.k, self.v):
            x.transpose(0, 2, 1, 3)[~owned] = np.nan
        self.masks = rng.integers(0, 2 ** 64, (B, T), dtype=np.uint64)  # bits behind a tree mean nothing
        if not empty_rows:
            self.masks |= np.uint64(1) << np.arange(T, dtype=np.uint64)
        else:
            self.masks[:, ::3] &= ~np.uint64(0) << np.uint64(T) if T < 64 else np.uint64(0)
        self.scale = D ** -0.5
        self.max_ctx = self.table.shape[1] * 16

    def run(self, kvc, out_dtype=torch.float16, **change):
        B = len(self.ctx)
        self.d = {**{x: dev(getattr(self, x)) for x in ("q", "k", "v", "table", "ctx")},
                  "masks": dev(self.masks.view(np.int64)), "lens": dev(self.lens), **change}
        d = self.d
        self.out = torch.full(self.q.shape, 55.0, dtype=out_dtype, device="cuda")
        need = kvc.paged_decode_tree_plan(B, self.Hq, self.Hkv, self.D, self.max_ctx, self.T)
        self.ws = torch.full((max(need, 16),), 0x7F, dtype=torch.uint8, device="cuda")
        self.call = kvc.paged_decode_tree_attention(d["q"], d["k"], d["v"], d["table"], d["ctx"], d["masks"], self.scale,
                                                    self.out, self.ws, self.max_ctx,
                                                    tree_lens=d["lens"], prepare=True)
        self.call()
        torch.cuda.synchronize()
        return host(self.out).astype(np.float64)

    def check(self, got, out_dtype, what="", rows=None):
        ref, spread = tree.tree_attention(self.q, self.k, self.v, self.table, self.ctx, self.masks, self.lens, self.scale)
        live = np.arange(self.T)[None] < self.lens[:, None]
        assert (got[~live] == 55.0).all(), f"{what}: a row behind a tree was written"
        if rows is not None:
            live &= rows
        got, ref, spread = got[live], ref[live], spread[live]
        if not got.size:
            return
        assert np.isfinite(got).all(), what
        N = int(self.ctx.max())
        half = out_dtype == torch.float16
        # scores: D products of at most |q||k| in fp32, scaled; |q k| scale stays below 8 sigma of sharp
        qk = np.abs(self.q.astype(np.float64)).max() * np.nanmax(np.abs(self.k.astype(np.float64))) * abs(self.scale)
        weight = (2.0 ** -11 if half else 2.0 ** -22) + self.D * 2.0 ** -24 * qk + 2.0 ** -21 + N * 2.0 ** -24
        # a weight below fp16's normal range keeps 2^-25 of the largest one; numerator and sum, hence twice
        small = 2 * N * 2.0 ** -25 * np.nanmax(np.abs(self.v.astype(np.float64)))
        bound = 2 * weight * spread + small + ((2.0 ** -11 if half else 2.0 ** -24) * np.abs(ref) + 2.0 ** -25)
        err = np.abs(got - ref)
        assert (err <= bound).all(), f"{what}: {np.nanmax(err / bound):.3f} of the bound, {int((err > bound).sum())} outputs"


TREES = [
    # hist, tree lens, T, Hq, Hkv, D, rows that see nothing
    ([0], [1], 1, 1, 1, 64, False),
    ([0, 5, 0], [4, 3, 0], 4, 4, 2, 64, True),
    ([127, 128, 120, 1, 15], [1, 1, 8, 7, 8], 8, 14, 2, 64, False),
    ([0, 64, 100, 191, 250], [64, 64, 33, 64, 1], 64, 2, 2, 64, True),
    ([300, 0, 77], [16, 16, 5], 16, 14, 2, 64, False),
    ([60, 500], [40, 64], 64, 14, 2, 64, False),          # 448 rows: two pairs of row tiles
    ([200, 1000, 3], [33, 17, 9], 33, 16, 4, 128, True),  # 132 rows: one and two row tiles in a batch
    ([90, 130], [64, 48], 64, 8, 2, 128, False),
    ([20, 600], [2, 3], 3, 64, 1, 64, False),             # 64 query heads on one KV head
    ([4000, 100, 0, 2100], [12, 12, 12, 3], 12, 8, 1, 128, True),  # a split context
    ([5000, 2500], [8, 1], 8, 14, 2, 64, False),
    ([0, 0], [0, 0], 5, 4, 4, 64, False),
    ([30, 31, 32], [2, 2, 2], 2, 8, 8, 128, False),
    ([40, 3], [64, 50], 64, 64, 1, 64, False),            # 4096 query rows
    ([30000, 9000, 0], [5, 5, 5], 5, 2, 1, 64, False),    # several clusters of chunks, and their combine
    ([20000, 3], [33, 40], 40, 8, 1, 128, True),          # the same with two row tiles
]


@pytest.mark.parametrize("case", range(len(TREES)))
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
def test_tree_attention(kvc, case, out_dtype):
    hist, lens, T, Hq, Hkv, D, empty = TREES[case]
    w = Tree(case, hist, lens, T, Hq, Hkv, D, empty)
    kvc.kvc_set_checked_mode(case % 2 == 0)
    got = w.run(kvc, out_dtype)
    assert kvc.kvc_device_error_flags() == 0
    w.check(got, out_dtype, f"tree case {case}")


@pytest.mark.parametrize("scale", [-0.3, 0.0, 0.5])
def test_tree_attention_scales_and_peaks(kvc, scale):
    w = Tree(20, [700, 130, 0], [10, 9, 10], 10, 14, 2, 64, True, sharp=4.0)
    w.scale = scale
    w.check(w.run(kvc), torch.float16, f"scale {scale}")


MANY = [
    # sequences, T, Hq, Hkv, D, histories up to, trees of nothing among them: more units than SMs
    (45, 9, 8, 8, 64, 300, 0),
    (100, 40, 14, 2, 64, 200, 0),      # 280 rows: pairs of two and of one row tile
    (60, 33, 16, 4, 128, 400, 0),      # 132 rows
    (90, 64, 8, 2, 128, 700, 0),
    (300, 3, 4, 2, 64, 60, 0),
    (1000, 2, 2, 1, 64, 40, 960),      # long runs of empty trees between units
    (40, 12, 32, 8, 128, 1500, 3),
]


def many(case, T, Hq, Hkv, D, B, far, none, empty=True):
    rng = np.random.default_rng([54, case])
    hist, lens = rng.integers(0, far + 1, B), rng.integers(1, T + 1, B)
    lens[rng.permutation(B)[:none]] = 0
    lens[0], hist[1 % B], hist[2 % B] = T, 0, far
    return Tree(100 + case, hist, lens, T, Hq, Hkv, D, empty)


@pytest.mark.parametrize("case", range(len(MANY)))
@pytest.mark.parametrize("out_dtype", [torch.float16, torch.float32])
def test_tree_attention_of_more_units_than_sms(kvc, case, out_dtype):
    B, T, Hq, Hkv, D, far, none = MANY[case]
    w = many(case, T, Hq, Hkv, D, B, far, none)
    got = w.run(kvc, out_dtype)
    assert kvc.kvc_device_error_flags() == 0
    w.check(got, out_dtype, f"many units, case {case}")
    again = w.run(kvc, out_dtype)
    assert (again == got).all()


@pytest.mark.parametrize("T,Hq,Hkv,D", [(6, 8, 8, 64), (40, 14, 2, 64), (20, 16, 2, 128)])
def test_many_units_with_bad_ones_among_them(kvc, T, Hq, Hkv, D):
    """Lengths that do not fit, block ids out of range, infinities and NaN in V rows of nodes: of the sequences they are
    in, not of the others that the same CTAs take."""
    B = 700 // Hkv
    w = many(20, T, Hq, Hkv, D, B, 150, 0, empty=False)
    w.masks[:] = np.uint64(1) << np.arange(T, dtype=np.uint64)  # each node sees itself alone, and the history
    w.lens[:], w.ctx[:] = np.minimum(w.lens, T), w.ctx
    good = w.run(kvc)
    bad_ctx, bad_table, pick = w.ctx.copy(), w.table.copy(), np.random.default_rng(7).permutation(B)
    short, block, inf = pick[:9], pick[9:20], pick[20:50]
    bad_ctx[short] = w.lens[short] - 1
    bad_table[block, 0] = len(w.k)
    v = w.v.copy()
    for b in inf:
        p = int(w.ctx[b] - 1)
        v[w.table[b][p // 16], :, p % 16, 5] = np.inf
    got = w.run(kvc, ctx=dev(bad_ctx), table=dev(bad_table), v=dev(v))
    assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["CONTEXT"] | kvc.DEVERR["BLOCK_ID"]
    for b in range(B):
        L = int(w.lens[b])
        if b in short or b in block:
            assert (got[b, :L] == 0).all(), b
        else:
            want = good[b].copy()
            if b in inf:
                want[L - 1, :, 5] = np.inf
            assert (got[b] == want).all(), b


def test_tree_of_a_chain_is_the_multi_token_decode(kvc):
    wl = workloads.multi_token_decode(21, [8, 40, 900], 8)
    d = [dev(x) for x in (wl.q, wl.k_pool, wl.v_pool, wl.block_table, wl.ctx)]
    B, most = 3, wl.block_table.shape[1] * 16
    outs = []
    for plan in (kvc.paged_decode_multi_plan, kvc.paged_decode_tree_plan):
        ws = torch.empty(max(16, plan(B, wl.Hq, wl.Hkv, wl.D, most, 8)), dtype=torch.uint8, device="cuda")
        out = torch.empty(wl.q.shape, dtype=torch.float32, device="cuda")
        if plan is kvc.paged_decode_multi_plan:
            kvc.paged_decode_multi_attention(*d, wl.scale, out, ws, most)
        else:
            masks = dev(kvc.kv_tree_masks(np.tile(np.arange(-1, 7, dtype=np.int32), (3, 1)))[0])
            kvc.paged_decode_tree_attention(*d, masks, wl.scale, out, ws, most)
        outs.append(out)
    # the multi-token decode's weights are rounded to fp16: 2^-11 on numerator and sum, of values up to ~5
    assert (outs[0] - outs[1]).abs().max().item() < 2 * 2.0 ** -11 * 5


@pytest.mark.parametrize("D,Hq,Hkv,T,hist", [(64, 14, 2, 12, 100), (128, 8, 2, 64, 200), (64, 4, 4, 40, 2000)])
def test_nodes_a_row_does_not_see_cannot_reach_it(kvc, D, Hq, Hkv, T, hist):
    """Infinities and NaN in K and V rows of nodes: rows that do not see them are as if they were zeros; rows that see
    a V infinity get it."""
    w = Tree(22, [hist], [T], T, Hq, Hkv, D)
    w.masks[:] = np.uint64(1) << np.arange(T, dtype=np.uint64)  # each node sees itself alone, and the history
    bad_nodes, inf_node = [3, T // 2], T - 1
    clean = w.run(kvc)

    def row_of(c, node):
        p = hist + node
        return c[w.table[0][p // 16], :, p % 16]
    for n in bad_nodes:
        row_of(w.k, n)[:] = np.nan
        row_of(w.v, n)[:] = np.nan
    row_of(w.v, inf_node)[:, 0] = np.inf
    row_of(w.v, inf_node)[:, D - 1] = -np.inf
    got = w.run(kvc)
    rest = [t for t in range(T) if t not in bad_nodes + [inf_node]]
    assert (got[0, rest] == clean[0, rest]).all()
    assert np.isnan(got[0, bad_nodes]).all()
    assert (got[0, inf_node, :, 0] == np.inf).all() and (got[0, inf_node, :, D - 1] == -np.inf).all()
    assert (got[0, inf_node, :, 1:D - 1] == clean[0, inf_node, :, 1:D - 1]).all()


def test_tree_attention_flags_bad_inputs(kvc):
    w = Tree(23, [300, 2500, 40, 100], [6, 6, 6, 6], 6, 14, 2, 64)
    good = w.run(kvc)
    bad_ctx, bad_len, bad_table = w.ctx.copy(), w.lens.copy(), w.table.copy()
    bad_ctx[0] = 3          # shorter than its tree
    bad_len[2] = 65         # no such tree
    got = w.run(kvc, ctx=dev(bad_ctx), lens=dev(bad_len))
    assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["CONTEXT"]
    assert (got[[0, 2]] == 0).all() and (got[[1, 3]] == good[[1, 3]]).all()
    bad_ctx = w.ctx.copy()
    bad_ctx[3] = w.max_ctx + 1
    assert (w.run(kvc, ctx=dev(bad_ctx))[3] == 0).all()
    assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["CONTEXT"]
    bad_table[1, 7] = len(w.k)
    bad_table[3, 0] = -1
    got = w.run(kvc, table=dev(bad_table))
    assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["BLOCK_ID"]
    assert np.isfinite(got).all() and (got[[0, 2]] == good[[0, 2]]).all() and (got[3] == 0).all()
    kvc.kvc_set_checked_mode(True)
    for change, name in ((dict(table=dev(bad_table)), "INVALID"), (dict(ctx=dev(bad_ctx)), "CAPACITY"),
                         (dict(lens=dev(bad_len)), "INVALID")):
        with pytest.raises(kvc.KvcError) as e:
            w.run(kvc, **change)
        assert e.value.name == "KVC_ERR_" + name


def test_tree_attention_argument_checks(kvc, monkeypatch):
    w = Tree(24, [30000], [4], 4, 4, 2, 64)
    w.run(kvc)
    d = w.d
    args = [d["q"], d["k"], d["v"], d["table"], d["ctx"], d["masks"], w.scale, w.out, w.ws, w.max_ctx]

    def call(i, x, **kw):
        return kvc.paged_decode_tree_attention(*args[:i], x, *args[i + 1:], **kw)
    for i, x, err in ((0, d["q"].float(), TypeError), (0, d["q"].transpose(1, 2).contiguous().transpose(1, 2), ValueError),
                      (5, d["masks"][:, :2], ValueError), (5, d["masks"].int(), TypeError), (7, w.out[:, :2], ValueError),
                      (7, w.out.to(torch.bfloat16), TypeError), (0, d["q"].cpu(), ValueError)):
        with pytest.raises(err):
            call(i, x)
    assert kvc.paged_decode_tree_plan(1, 4, 2, 64, w.max_ctx, 4) > 0
    for ws in (None, w.ws[:-16], w.ws[8:]):
        with pytest.raises(kvc.KvcError) as e:
            call(8, ws)
        assert e.value.name == "KVC_ERR_INVALID"
    monkeypatch.setattr(kvc, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        call(0, d["q"])


def test_tree_attention_captured_on_another_stream(kvc):
    """A captured call follows the lengths, masks and queries it finds at replay; two graphs share a workspace."""
    w, x = Tree(25, [30000, 50], [9, 20], 20, 14, 2, 64), Tree(26, [10, 10], [20, 3], 20, 14, 2, 64)
    x.table, x.k, x.v, x.max_ctx = w.table, w.k, w.v, w.max_ctx
    x.ctx = np.array([30005, 60], np.int32)  # inside what the pool holds
    assert kvc.paged_decode_tree_plan(2, 14, 2, 64, w.max_ctx, 20) > 0
    ref = []
    for t in (w, x):
        t.check(t.run(kvc), torch.float16)
        ref.append(host(t.out))
    s = torch.cuda.Stream()
    graphs = []
    for t in (w, x):
        args = [t.d[k] for k in ("q", "k", "v", "table", "ctx", "masks")]
        out = torch.full_like(t.out, 55.0)
        kvc.paged_decode_tree_attention(*args, t.scale, out, w.ws, t.max_ctx, tree_lens=t.d["lens"], stream=s)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            kvc.paged_decode_tree_attention(*args, t.scale, out, w.ws, t.max_ctx, tree_lens=t.d["lens"])
        graphs.append((g, out))
    for _ in range(3):
        for (g, out), r in zip(graphs, ref):
            out.fill_(55.0)
            g.replay()
        torch.cuda.synchronize()
        for (g, out), r in zip(graphs, ref):
            assert (host(out) == r).all()
    for name in ("q", "ctx", "masks", "lens"):  # the first graph with the second's inputs
        w.d[name].copy_(x.d[name])
    graphs[0][1].fill_(55.0)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert (host(graphs[0][1]) == ref[1]).all()


# ---------------------------------------------------------------- verification
def verify_case(seed, B, T, V, noise=0.7, half=False, distinct=False, temp=2.0, parents=None):
    """Rows of probabilities, a tree drawn from the draft's, uniforms."""
    rng = np.random.default_rng([53, seed])
    par = np.full((B, T), -1, np.int32)
    for t in range(1, T):
        par[:, t] = rng.integers(max(0, t - 5), t, B) if parents is None else parents[t]
    x = temp * rng.standard_normal((B, T, V))
    y = x + noise * rng.standard_normal((B, T, V))
    soft = lambda z: np.exp(z - z.max(-1, keepdims=True)) / np.exp(z - z.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
    dt = np.float16 if half else np.float32
    p, q = soft(x).astype(dt), soft(y).astype(dt)
    tok = np.zeros((B, T), np.int32)
    for b in range(B):
        for t in range(1, T):
            w = q[b, par[b, t]].astype(np.float64)
            if distinct:
                w[[tok[b, s] for s in range(1, t) if par[b, s] == par[b, t]]] = 0
            c = np.cumsum(w)
            tok[b, t] = min(V - 1, np.searchsorted(c, rng.random() * c[-1], side="right"))
    return p, q, tok, par, rng.random((B, T), dtype=np.float32)


def run_verify(kvc, p, q, tok, par, u, lens=None, distinct=False, stream=None):
    B, T = tok.shape
    path = torch.full((B, T), 77, dtype=torch.int32, device="cuda")
    n, nxt = (torch.full((B,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    as_dev = lambda a: a if isinstance(a, torch.Tensor) else dev(a)  # noqa: E731
    kvc.draft_tree_verify(as_dev(p), as_dev(q), dev(tok), dev(par), dev(u), path, n, nxt,
                          tree_lens=None if lens is None else dev(lens), distinct=distinct, stream=stream)
    torch.cuda.synchronize()
    return host(path), host(n), host(nxt)


def check_verify(got, p, q, tok, par, u, lens=None, distinct=False):
    path, n, nxt = got
    for b in range(len(tok)):
        L = tok.shape[1] if lens is None else int(lens[b])
        if L == 0:
            assert n[b] == 0 and nxt[b] == -1 and (path[b] == -1).all()
            continue
        want, token = tree.verify(p[b, :L], q[b, :L], tok[b, :L], par[b, :L], u[b, :L].astype(np.float64), distinct)
        assert n[b] == len(want) and path[b, :n[b]].tolist() == want and (path[b, n[b]:] == -1).all(), (b, path[b], want)
        assert nxt[b] == token, (b, nxt[b], token)


VERIFY = [
    # B, T, V, noise, fp16, distinct
    (3, 1, 1, 0.7, False, False),
    (40, 4, 7, 0.7, False, False),
    (40, 9, 33, 1.5, False, True),
    (20, 64, 501, 1.0, False, True),
    (20, 64, 501, 0.3, True, False),
    (8, 12, 1025, 0.7, True, True),
    (5, 8, 32000, 0.7, False, False),
    (6, 6, 50001, 2.0, False, True),
    (3, 5, 128257, 1.0, False, False),
    (2, 4, 200003, 1.0, True, True),
]


@pytest.mark.parametrize("case", range(len(VERIFY)))
def test_verify(kvc, case):
    B, T, V, noise, half, distinct = VERIFY[case]
    p, q, tok, par, u = verify_case(case, B, T, V, noise, half, distinct and V > T)
    kvc.kvc_set_checked_mode(case % 2 == 0)
    first = run_verify(kvc, p, q, tok, par, u, distinct=distinct)
    assert kvc.kvc_device_error_flags() == 0
    check_verify(first, p, q, tok, par, u, distinct=distinct)
    again = run_verify(kvc, p, q, tok, par, u, distinct=distinct)
    assert all((a == b).all() for a, b in zip(first, again))


MANY_VERIFY = [
    # B, T, V, fp16, distinct: clusters of other sizes than a few sequences get
    (64, 2, 128257, False, False),
    (19, 3, 128257, False, True),
    (30, 3, 90001, True, False),
    (130, 2, 60007, False, False),
    (160, 3, 30011, True, True),
    (500, 4, 601, False, True),
    (200, 3, 9001, False, False),
]


@pytest.mark.parametrize("case", range(len(MANY_VERIFY)))
def test_verify_of_many_sequences(kvc, case):
    B, T, V, half, distinct = MANY_VERIFY[case]
    p, q, tok, par, u = verify_case(70 + case, B, T, V, 1.5, half, distinct, parents=[0] * T)
    u[:, 1:] = np.minimum(1 - u[:, 1:] * 0.3, np.float32(1 - 2.0 ** -24))  # refusals
    got = run_verify(kvc, p, q, tok, par, u, distinct=distinct)
    assert kvc.kvc_device_error_flags() == 0
    check_verify(got, p, q, tok, par, u, distinct=distinct)
    assert (got[1] == 1).any() and (got[1] > 1).any()
    assert all((a == b).all() for a, b in zip(got, run_verify(kvc, p, q, tok, par, u, distinct=distinct)))


@pytest.mark.parametrize("distinct", [False, True])
def test_verify_many_refusals_at_one_node(kvc, distinct):
    """All nodes are the root's children, under uniforms near 1, so that most are refused; the same token twice."""
    T, V = 20, 97
    p, q, tok, par, u = verify_case(60, 32, T, V, 2.0, distinct=distinct, parents=[0] * T)
    u[:, 1:] = 1 - u[:, 1:] * 0.05
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    if not distinct:
        tok[:, 5] = tok[:, 4]
    got = run_verify(kvc, p, q, tok, par, u, distinct=distinct)
    check_verify(got, p, q, tok, par, u, distinct=distinct)


@pytest.mark.parametrize("T,V,parents", [(20, 97, "root"), (64, 40, "root"), (64, 33, "random"), (33, 5, "random")])
def test_verify_distinct_children_with_a_token_twice(kvc, T, V, parents):
    """A token that was refused at a node has no mass in the draft's row there any more: trying it again refuses it
    and takes no further mass."""
    par = [0] * T if parents == "root" else None
    p, q, tok, par, u = verify_case(61 + T + V, 32, T, V, 2.0, parents=par)  # drawn with replacement: tokens repeat
    u[:, 1:] = 1 - u[:, 1:] * 0.05
    u = np.minimum(u, np.float32(1 - 2.0 ** -24))
    assert any(len(set(tok[b, 1:][par[b, 1:] == 0])) < (par[b, 1:] == 0).sum() for b in range(32))
    got = run_verify(kvc, p, q, tok, par, u, distinct=True)
    check_verify(got, p, q, tok, par, u, distinct=True)


def test_verify_ragged_trees_and_strided_rows(kvc):
    B, T, V = 9, 10, 700
    p, q, tok, par, u = verify_case(61, B, T, V)
    lens = np.array([10, 0, 1, 2, 5, 9, 10, 3, 7], np.int32)
    wide_p, wide_q = (torch.full((B, T, w), float("nan"), device="cuda") for w in (V + 3, V + 64))
    wide_p[..., :V], wide_q[..., :V] = dev(p), dev(q)
    got = run_verify(kvc, wide_p[..., :V], wide_q[..., :V], tok, par, u, lens)
    check_verify(got, p, q, tok, par, u, lens)
    assert kvc.kvc_device_error_flags() == 0


def test_verify_edges(kvc):
    V = 600
    p, q, tok, par, u = verify_case(62, 6, 4, V)
    u[0] = 0.0                                         # everything with mass is kept; the draw takes the first entry
    p[0, :, :5] = 0.0
    tok[0] = 9
    q[1] = p[1]                                        # the draft is the target
    p[2], q[2] = 0.0, 0.0                              # greedy rows: one token holds everything
    p[2, :, 17], q[2, :, 17] = 1.0, 1.0
    tok[2] = 17
    p[3], q[3] = 0.0, 0.0                              # the draft sure of a token that the target never takes
    p[3, :, 400], q[3, :, 3] = 1.0, 1.0
    tok[3] = 3
    u[4] = 1 - 2.0 ** -24
    q[5, :, 100:] = np.nan                             # NaN and negative values count as nothing
    p[5, :, 50:60] = -1.0
    tok[5] = 20
    got = run_verify(kvc, p, q, tok, par, u)
    assert kvc.kvc_device_error_flags() == 0
    p, q = (np.nan_to_num(x).clip(0) for x in (p, q))
    check_verify(got, p, q, tok, par, u)
    assert got[2][0] == 5 and got[2][3] == 400 and got[2][2] == 17 and got[1][2] > 1 and got[1][3] == 1


def test_verify_captured_beside_another(kvc):
    """Two captured calls replayed at once on two streams (the call has no workspace), with new uniforms each time."""
    cases = [verify_case(70 + i, 8, 10, 4001, 1.0, distinct=bool(i)) for i in range(2)]
    runs = []
    for i, (p, q, tok, par, u) in enumerate(cases):
        s = torch.cuda.Stream()
        d = [dev(x) for x in (p, q, tok, par, u)]
        out = [torch.zeros(8, 10, dtype=torch.int32, device="cuda")] + [torch.zeros(8, dtype=torch.int32, device="cuda")
                                                                       for _ in range(2)]
        call = kvc.draft_tree_verify(*d, *out, distinct=bool(i), prepare=True)
        s.wait_stream(torch.cuda.current_stream())
        call(s)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
        runs.append((g, s, d, out))
    for turn in range(3):
        us = []
        for i, (g, s, d, out) in enumerate(runs):
            us.append(np.random.default_rng(100 * turn + i).random((8, 10), dtype=np.float32))
            d[4].copy_(dev(us[-1]))
        torch.cuda.synchronize()
        for g, s, d, out in runs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i, (g, s, d, out) in enumerate(runs):
            p, q, tok, par, _ = cases[i]
            check_verify([host(x) for x in out], p, q, tok, par, us[i], distinct=bool(i))


def test_verify_flags_bad_trees(kvc):
    p, q, tok, par, u = verify_case(63, 5, 4, 50)
    tok0, par0 = tok.copy(), par.copy()
    tok[0, 1], tok[1, 2], par[2, 3], par[3, 1] = 50, -1, 3, -1
    got = run_verify(kvc, p, q, tok, par, u)
    assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["TREE"]
    par2 = par.copy()
    for b, t in ((0, 1), (1, 2), (2, 3), (3, 1)):
        par2[b, t] = -2  # such a node is nobody's child
    check_verify(got, p, q, np.clip(tok, 0, 49), par2, u)
    got = run_verify(kvc, np.zeros_like(p), q, tok0, par0, u)  # rows without mass
    assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["TREE"]
    assert (got[2] == -1).all() and (got[1] == 1).all()
    got = run_verify(kvc, p, q, tok0, par0, u, np.array([4, 5, -1, 4, 0], np.int32))
    assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["TREE"]
    check_verify(got, p, q, tok0, par0, u, np.array([4, 0, 0, 4, 0]))
    kvc.kvc_set_checked_mode(True)
    with pytest.raises(kvc.KvcError):
        run_verify(kvc, p, q, tok, par, u)
    with pytest.raises(ValueError):
        run_verify(kvc, p, q[:, :, :40], tok0, par0, u)
    with pytest.raises(ValueError):
        run_verify(kvc, dev(p).transpose(0, 1).contiguous().transpose(0, 1), q, tok0, par0, u)


# ---------------------------------------------------------------- commit
def commit_case(seed, L, hist, lens, T, Hkv, D):
    rng = np.random.default_rng([54, seed])
    lens = np.array(lens, np.int32)
    ctx = (np.array(hist) + lens).astype(np.int32)
    nblk = [-(-int(c) // 16) for c in ctx]
    NB = sum(nblk) + 1
    perm = rng.permutation(NB).astype(np.int32)
    table, at = np.full((len(ctx), max(nblk)), -3, np.int32), 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n]
        at += n
    path, n = np.full((len(ctx), T), -1, np.int32), np.zeros(len(ctx), np.int32)
    for b, ln in enumerate(lens):
        if ln:
            rest = np.sort(rng.permutation(np.arange(1, ln))[:rng.integers(0, ln)])
            n[b] = 1 + len(rest)
            path[b, :n[b]] = np.concatenate([[0], rest])
    pools = [rng.integers(0, 2 ** 16, (L, NB, Hkv, 16, D), dtype=np.uint16).view(np.float16) for _ in range(2)]
    return pools, table, ctx, lens, path, n


@pytest.mark.parametrize("L,hist,lens,T,Hkv,D", [
    (1, [0], [1], 1, 1, 64), (3, [5, 100, 0, 33], [8, 8, 8, 3], 8, 2, 64), (24, [15, 16, 17], [64, 40, 0], 64, 8, 128),
    (2, [1000] * 70, list(range(70 - 64, 70 - 6)) + [64] * 12, 64, 4, 64), (1, [3], [64], 64, 64, 128)])
def test_commit(kvc, L, hist, lens, T, Hkv, D):
    pools, table, ctx, lens, path, n = commit_case(len(hist) + L, L, hist, lens, T, Hkv, D)
    d = [dev(p.view(np.int16)).view(torch.float16) for p in pools]
    h = kvc.kv_cache_create(kvc.KvcConfig(L, pools[0].shape[1], Hkv, D), *d)
    try:
        for mode in (False, True):
            kvc.kvc_set_checked_mode(mode)
            new = torch.full((len(ctx),), 99, dtype=torch.int32, device="cuda")
            kvc.kv_tree_commit(h, dev(table), dev(ctx), dev(path), dev(n), new, tree_lens=dev(lens))
            torch.cuda.synchronize()
            want = tree.commit(pools, table, ctx, lens, path, n)
            assert kvc.kvc_device_error_flags() == 0
            assert (host(new) == want).all()
            for got, ref in zip(d, pools):
                assert (host(got).view(np.uint16) == ref.view(np.uint16)).all()
    finally:
        kvc.kv_cache_destroy(h)


def test_commit_of_a_path_narrower_than_its_tree(kvc):
    """A tree of 40 nodes whose depth is known to be at most 5: the path is [B][5]."""
    pools, table, ctx, lens, path, n = commit_case(77, 2, [50, 9], [40, 33], 40, 2, 64)
    path, n = np.array([[0, 3, 7, 20, 39], [0, 1, 32, -1, -1]], np.int32), np.array([5, 3], np.int32)
    d = [dev(p.view(np.int16)).view(torch.float16) for p in pools]
    h = kvc.kv_cache_create(kvc.KvcConfig(2, pools[0].shape[1], 2, 64), *d)
    try:
        new = torch.zeros(2, dtype=torch.int32, device="cuda")
        kvc.kv_tree_commit(h, dev(table), dev(ctx), dev(path), dev(n), new, tree_lens=dev(lens))
        assert (host(new) == tree.commit(pools, table, ctx, lens, path, n)).all()
        for got, ref in zip(d, pools):
            assert (host(got).view(np.uint16) == ref.view(np.uint16)).all()
    finally:
        kvc.kv_cache_destroy(h)


def test_commit_flags_bad_inputs_and_leaves_the_sequence(kvc):
    L, T = 2, 8
    pools, table, ctx, lens, path, n = commit_case(9, L, [20] * 9, [8] * 9, T, 2, 64)
    path[:], n[:] = -1, 3
    path[:, :3] = [0, 4, 7]
    d = [dev(p.view(np.int16)).view(torch.float16) for p in pools]
    h = kvc.kv_cache_create(kvc.KvcConfig(L, pools[0].shape[1], 2, 64), *d)
    good = [path.copy(), n.copy(), ctx.copy(), table.copy()]
    try:
        path[0, :3], path[1, :3], path[2, :3], path[3, 0] = [0, 4, 4], [0, 4, 8], [0, -2, 3], 1  # not an increasing path
        n[4] = 9
        ctx[5] = 5             # shorter than its tree
        ctx[6] = 16 * table.shape[1] + 1
        table[7, 1] = 10 ** 6  # the block of positions 16 .. 31
        new = torch.zeros(9, dtype=torch.int32, device="cuda")
        kvc.kv_tree_commit(h, dev(table), dev(ctx), dev(path), dev(n), new, tree_lens=dev(lens))
        E = kvc.DEVERR
        assert kvc.kvc_device_error_flags(clear=True) == E["TREE"] | E["CONTEXT"] | E["BLOCK_ID"]
        want = ctx.copy()
        want[8:] = tree.commit(pools, table[8:], ctx[8:], lens[8:], path[8:], n[8:])
        assert (host(new) == want).all()
        for got, ref in zip(d, pools):
            assert (host(got).view(np.uint16) == ref.view(np.uint16)).all()
        kvc.kvc_set_checked_mode(True)
        for i, names in ((0, "INVALID"), (4, "INVALID"), (5, "CAPACITY"), (6, "CAPACITY"), (7, "INVALID")):
            pa, nn, cc, tt = (x.copy() for x in good)
            pa[i], nn[i], cc[i], tt[i] = path[i], n[i], ctx[i], table[i]
            with pytest.raises(kvc.KvcError) as e:
                kvc.kv_tree_commit(h, dev(tt), dev(cc), dev(pa), dev(nn), new, tree_lens=dev(lens))
            assert e.value.name == "KVC_ERR_" + names
    finally:
        kvc.kv_cache_destroy(h)


# ---------------------------------------------------------------- the operators together
def reference_step(wl):
    """The whole step in fp64 on the host: rotated rows rounded to fp16 where the cache holds them."""
    B, T = wl.parents.shape
    masks, depths = tree.tree_masks(wl.parents, wl.tree_lens)
    angle = ((wl.hist[:, None] + depths).reshape(-1, 1) * wl.inv_freq).astype(np.float64)
    pools = [wl.k_pool.copy(), wl.v_pool.copy()]
    qs = []
    for lay in range(wl.L):
        q, k, v = np.split(wl.qkv[lay].reshape(B * T, -1, wl.D), [wl.Hq, wl.Hq + wl.Hkv], 1)
        qs.append(tree.norm_rotate(q, wl.q_weight[lay], wl.eps, angle, False).astype(np.float16).reshape(B, T, wl.Hq, wl.D))
        k = tree.norm_rotate(k, wl.k_weight[lay], wl.eps, angle, False).astype(np.float16)
        for b in range(B):
            for t in range(int(wl.tree_lens[b])):
                pos = int(wl.hist[b]) + t
                for pool, rows in zip(pools, (k, v)):
                    pool[lay, wl.block_table[b, pos // 16], :, pos % 16] = rows[b * T + t]
    return masks, qs, pools


def test_a_whole_step_then_an_ordinary_decode(kvc):
    """Two layers of append and attention, verification, commit, all replayed from one graph; the committed context is
    then decoded like any other and matches the sequence of kept tokens built from scratch."""
    from paged_kv_cache_27_gb300.harness import TreeSession
    import oracle
    wl = workloads.tree_decode(1, [0, 15, 100, 700, 33], [12, 1, 12, 7, 0], 12, L=2)
    s = TreeSession(wl)
    s.step()
    torch.cuda.synchronize()
    for p, init in ((s.k_pool, wl.k_pool), (s.v_pool, wl.v_pool)):
        p.copy_(dev(init))
    s.out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    g.replay()
    torch.cuda.synchronize()
    assert kvc.kvc_device_error_flags() == 0
    masks, qs, pools = reference_step(wl)
    for lay in range(wl.L):
        ref, spread = tree.tree_attention(qs[lay], pools[0][lay], pools[1][lay], wl.block_table, wl.ctx, masks,
                                          wl.tree_lens, wl.scale)
        live = np.arange(wl.T)[None] < wl.tree_lens[:, None]
        got = host(s.out[lay]).astype(np.float64)
        assert (got[~live] == 0).all()
        # one fp16 step of the query and of the keys (the reference's own roundings), scores of size |q||k| scale,
        # and the attention's weights; a score error e changes an output by 2 e spread
        qk = np.abs(qs[lay].astype(np.float64)).max() * np.abs(pools[0][lay].astype(np.float64)).max() * wl.scale
        bound = 2 * (2.0 ** -10 * qk * np.sqrt(wl.D) + 2.0 ** -11) * spread + 2.0 ** -11 * np.abs(ref) + 2e-4
        assert (np.abs(got - ref)[live] <= bound[live]).all()
    walks = [tree.verify(wl.p[b, :n], wl.q[b, :n], wl.tokens[b, :n], wl.parents[b, :n],
                         wl.uniforms[b, :n].astype(np.float64), False) if n else ([], -1)
             for b, n in enumerate(wl.tree_lens)]
    assert host(s.path_len).tolist() == [len(w[0]) for w in walks]
    assert host(s.next_token).tolist() == [w[1] for w in walks]
    for b, (walk, _) in enumerate(walks):
        assert host(s.path)[b, :len(walk)].tolist() == walk
    new_ctx = wl.hist + np.array([len(w[0]) for w in walks], np.int32)
    assert (host(s.new_context_lens) == new_ctx).all()
    # the committed rows are the kept nodes' own: history, then the path, gathered from scratch
    for lay in range(wl.L):
        for pool, got in zip(pools, (s.k_pool, s.v_pool)):
            for b, (walk, _) in enumerate(walks):
                rows = tree.rows_of(pool[lay], wl.block_table[b], int(wl.ctx[b]))
                want = np.concatenate([rows[:wl.hist[b]], rows[wl.hist[b]:][walk]]) if walk else rows[:wl.hist[b]]
                have = tree.rows_of(host(got[lay]), wl.block_table[b], int(new_ctx[b]))
                # keys differ by their own fp16 rounding where the fp32 value sits between two
                assert np.abs(have.astype(np.float64) - want).max(initial=0) <= 2.0 ** -10 * np.abs(want).max(initial=1)
    keep = new_ctx > 0
    q = dev(workloads.normal_f16(np.random.default_rng(1), (int(keep.sum()), wl.Hq, wl.D)))
    table, ctx = dev(wl.block_table[keep]), s.new_context_lens[dev(np.flatnonzero(keep))].contiguous()
    _, _, need = kvc.paged_decode_plan(len(q), wl.Hq, wl.Hkv, wl.D, s.max_ctx)
    out = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    kvc.paged_decode_attention(q, s.k_pool[1], s.v_pool[1], table, ctx, wl.scale, out,
                               torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"), s.max_ctx)
    ref = oracle.decode(host(q), host(s.k_pool[1]), host(s.v_pool[1]), wl.block_table[keep], new_ctx[keep], wl.scale)
    assert np.abs(host(out) - ref).max() <= 2e-3
    s.close()


@pytest.mark.parametrize("graph", [False, True])
def test_calls_wait_for_the_kernel_in_front(kvc, graph):
    """Every call is launched as a programmatic dependent: what a kernel right in front of it writes is what it reads,
    and a buffer that the kernel in front still reads is not overwritten early."""
    from paged_kv_cache_27_gb300.harness import TreeSession
    wl = workloads.tree_decode(2, [40, 300, 7], [12, 9, 12], 12, L=2)
    s = TreeSession(wl)
    fresh = [x.clone() for x in (s.k_pool, s.v_pool)]
    results = lambda: [host(x) for x in (s.out, s.path, s.path_len, s.next_token, s.new_context_lens, s.k_pool, s.v_pool)]  # noqa: E731
    s.step()
    torch.cuda.synchronize()
    want = results()
    late = {0: s.qkv[0], 1: s.masks, 2: s.qkv[1], 3: s.tree_lens, 4: s.p, 5: s.block_table}  # of the calls in order
    right = {i: x.clone() for i, x in late.items()}
    big = torch.zeros(64 << 20, device="cuda")
    seen = torch.empty_like(s.q_rot[1])

    def step():
        for pool, x in zip((s.k_pool, s.v_pool), fresh):
            torch.add(x, 0, out=pool)
        for i, call in enumerate(s._calls):
            late[i].fill_(0)
            big.add_(1)  # long, so that its successors queue up
            torch.add(right[i], 0, out=late[i])
            call()
            if i == 2:
                torch.add(s.q_rot[1], 0, out=seen)
    step()
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        s.out.zero_()
        g.replay()
        torch.cuda.synchronize()
    assert kvc.kvc_device_error_flags() == 0
    for a, b in zip(results(), want):
        assert np.array_equal(a.view(np.uint8), b.view(np.uint8))
    assert (seen == s.q_rot[1]).all()
