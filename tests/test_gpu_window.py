"""Windows, the block-scaled cache and tables built on the GPU against their definitions in 64 bits.

Pools are poisoned: rows that no query may see hold NaN or infinities, table entries of blocks in which nothing is
visible hold ids out of range.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_27_gb300 as kvc
from oracle import window as ow

pytestmark = pytest.mark.gpu
BS = 16
HEADS = [(14, 2, 64), (32, 8, 128), (3, 3, 64), (20, 1, 128), (12, 4, 64)]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(got, ref, top, vmax, n, D, extra=0.0):
    """got against ref within what the arithmetic allows: scores are sums of D fp32 products (the tensor cores' additions
    may cut off: a whole 2^-23 each), times scale and log2 e; a weight is off by its score's error, 2^-20 for 2^x and its
    two fp16 parts, and 2^-32 of the largest one; the sums of n / 16 tiles and the merges add 2^-23 each.  `top`: the
    largest sum of |q k scale| of a row; `extra`: a form's own rounding of weights.  An fp16 output adds half a step."""
    weight = np.expm1((D + 8) * 2.0 ** -23 * top) + 2.0 ** -20 + n * 2.0 ** -32 + extra
    tol = 2 * vmax * weight + (n / 8 + 64) * 2.0 ** -23 * vmax
    if got.dtype == torch.float16:
        tol = tol + (np.abs(ref) + tol) * 2.0 ** -11 + 2.0 ** -25
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    err = np.abs(g - ref)
    assert (err <= tol).all(), (err.max(), np.max(tol), np.unravel_index((err - tol).argmax(), err.shape))


class Case:
    """A paged cache of B sequences with the contexts ctx; what is not visible is poisoned."""

    def __init__(self, ctx, heads, window, sinks, fp8, seed=0, spread=0):
        self.ctx, self.window, self.sinks, self.fp8 = np.asarray(ctx, np.int32), window, sinks, fp8
        self.Hq, self.Hkv, self.D = heads
        rng = np.random.default_rng(seed)
        B, most = len(ctx), int(max(1, -(-max(ctx) // BS))) + 2
        self.NB = int(sum(-(-c // BS) for c in ctx)) + 3
        ids = rng.permutation(self.NB)
        self.table = rng.choice([-1, -7, self.NB, 2 ** 31 - 1], (B, most)).astype(np.int32)  # never followed
        self.q = rng.standard_normal((B, self.Hq, self.D)).astype(np.float16)
        shape = (self.NB, self.Hkv, 2, BS, self.D)
        seen = np.zeros((self.NB, BS), bool)
        at = 0
        for b, n in enumerate(self.ctx):
            for j in range(-(-int(n) // BS)):
                p = [p for p in range(j * BS, (j + 1) * BS) if p < n and (window == 0 or p >= n - window or p < sinks)]
                if p:
                    self.table[b, j] = ids[at]
                    seen[ids[at], [x % BS for x in p]] = True
                at += 1
        if fp8:
            e = rng.integers(-9 - spread, -6 + spread + 1, shape[:3])
            self.scales = (2.0 ** e).astype(np.float32)
            self.codes = rng.integers(0, 256, shape).astype(np.uint8)
            self.codes[(self.codes & 0x7f) == 0x7f] = 0x30
            codes = self.codes.copy()
            codes.transpose(0, 3, 1, 2, 4)[~seen] = 0x7f  # NaN
            scales = self.scales.copy()
            scales[~seen.any(1)] = np.nan
            self.cache = dev(codes), dev(scales)
            self.values = ow.e4m3_values(self.codes) * self.scales.astype(np.float64)[..., None, None]
        else:
            kv = rng.standard_normal(shape).astype(np.float16)
            self.values = kv.astype(np.float64)
            hidden = kv.transpose(0, 3, 1, 2, 4)
            hidden[~seen] = rng.choice([np.nan, np.inf, -np.inf], hidden[~seen].shape)
            self.cache = dev(kv[:, :, 0]), dev(kv[:, :, 1])

    def rows(self, b, p):
        x = self.values[self.table[b, p // BS], :, :, p % BS]  # [n][Hkv][2][D]
        return x[:, :, 0], x[:, :, 1]

    def reference(self, scale):
        ref = ow.decode(self.q, self.rows_of(), scale, self.window, self.sinks)
        return ref

    def rows_of(self):
        f = lambda b, p: self.rows(b, p)  # noqa: E731
        f.ctx = self.ctx
        return f

    def limits(self, scale):
        """The largest sum of |q k scale| of a row and the largest |v|."""
        top = vmax = 0.0
        for b in range(len(self.ctx)):
            k, v = self.rows(b, ow.visible(int(self.ctx[b]), self.window, self.sinks))
            for h in range(self.Hq):
                top = max(top, float((np.abs(k[:, h * self.Hkv // self.Hq]) @ np.abs(self.q[b, h].astype(np.float64))).max()))
            vmax = max(vmax, float(np.abs(v).max()))
        return top * abs(scale), vmax

    def run(self, scale, out, most=None, stream=None, prepare=False, **new):
        B, most = len(self.ctx), int(most or self.ctx.max())
        args = (dev(self.table), dev(self.ctx))
        if self.fp8:
            n = kvc.paged_decode_fp8_block_plan(B, self.Hq, self.Hkv, self.D, most, self.window, self.sinks)
            ws = torch.full((max(n, 16),), 0xff, dtype=torch.uint8, device="cuda")
            return kvc.paged_decode_attention_fp8_block(dev(self.q), *self.cache, *args, scale, out, ws, most, self.window,
                                                        self.sinks, stream=stream, prepare=prepare)
        n = kvc.paged_decode_window_plan(B, self.Hq, self.Hkv, self.D, most, self.window, self.sinks)
        ws = torch.full((max(n, 16),), 0xff, dtype=torch.uint8, device="cuda")
        return kvc.paged_decode_window_attention(dev(self.q), *self.cache, *args, self.window, self.sinks, scale, out, ws,
                                                 most, stream=stream, prepare=prepare, **new)

    def out(self, dtype=torch.float32):
        return torch.full((len(self.ctx), self.Hq, self.D), float("nan"), dtype=dtype, device="cuda")


CTX = [1, 15, 16, 17, 40, 100, 333, 32, 65]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (15, 1), (16, 4), (17, 16), (40, 33), (5, 7), (64, 0), (64, 90), (1000, 4),
                                          (1, 1000)])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_windows(heads, window, sinks, fp8):
    c = Case(CTX, heads, window, sinks, fp8, seed=window + sinks, spread=1)
    scale = heads[2] ** -0.5
    top, vmax = c.limits(scale)
    ref = c.reference(scale)
    for dtype in (torch.float32, torch.float16):
        out = c.out(dtype)
        c.run(scale, out)
        check(out, ref, top, vmax, 400, heads[2])
    assert kvc.kvc_device_error_flags(clear=True) == 0


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("scale", [0.125, -0.2, 0.0, 1.0])
def test_decode_of_the_whole_context(heads, scale):
    c = Case(CTX, heads, 0, 0, True, seed=3, spread=0)
    top, vmax = c.limits(scale)
    out = c.out()
    c.run(scale, out, most=352)
    check(out, c.reference(scale), top, vmax, 400, heads[2])
    assert kvc.kvc_device_error_flags(clear=True) == 0


@pytest.mark.parametrize("heads,ctx,window,sinks,fp8", [
    ((14, 2, 64), [40000], 0, 0, True), ((2, 1, 128), [70001, 3], 0, 0, True), ((14, 2, 64), [70000], 60001, 100, False),
    ((8, 1, 128), [30000, 29999, 7], 20000, 17, True), ((2, 2, 64), [5000] * 40, 3000, 4, False),
    ((2, 2, 64), [4000] * 70 + [17] * 30, 0, 0, True)])
def test_decode_of_long_contexts(heads, ctx, window, sinks, fp8):
    """Several clusters along a context (their parts merged by a second kernel), and more units than are resident."""
    c = Case(ctx, heads, window, sinks, fp8, seed=5)
    scale = heads[2] ** -0.5
    top, vmax = c.limits(scale)
    out = c.out()
    c.run(scale, out)
    check(out, c.reference(scale), top, vmax, max(ctx), heads[2])
    assert kvc.kvc_device_error_flags(clear=True) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_scales_far_apart(D):
    """V scales 2^-30 to 2^6 over one context, the largest weights on any of them."""
    for seed in range(4):
        c = Case([500, 90], (8, 2, D), 0, 0, True, seed=seed, spread=0)
        rng = np.random.default_rng(seed)
        e = rng.integers(-30, 7, c.scales[:, :, 1].shape)
        c.scales[:, :, 1] = 2.0 ** e
        c.values = ow.e4m3_values(c.codes) * c.scales.astype(np.float64)[..., None, None]
        c.cache = c.cache[0], dev(np.where(np.isnan(c.cache[1].cpu().numpy()), np.nan, c.scales).astype(np.float32))
        top, vmax = c.limits(0.5)
        out = c.out()
        c.run(0.5, out)
        check(out, c.reference(0.5), top, vmax, 500, D)
        # a context whose every scale is small keeps its digits
        c.scales[:, :, 1] = 2.0 ** -31
        c.values = ow.e4m3_values(c.codes) * c.scales.astype(np.float64)[..., None, None]
        c.cache = c.cache[0], dev(np.where(np.isnan(c.cache[1].cpu().numpy()), np.nan, c.scales).astype(np.float32))
        out = c.out()
        c.run(0.5, out)
        check(out, c.reference(0.5), top, 448 * 2.0 ** -31, 500, D)


@pytest.mark.parametrize("fp8", [False, True])
def test_weights_far_below_the_largest_keep_their_mass(fp8):
    """65,536 keys 17.4 nats below one of them: 1.8e-3 of the row."""
    n, D = 65537, 64
    c = Case([n], (1, 1, D), 0 if fp8 else 2 ** 30, 0, fp8, seed=9)
    c.q[:] = 0
    c.q[0, 0, 0] = 8
    k = np.zeros((c.NB, 1, BS, D))
    v = np.ones((c.NB, 1, BS, D))
    first = c.table[0, 100]
    k[first, 0, 5, 0], v[first, 0, 5] = 2.175, -1  # (e4m3: 2.25, fp16: 2.1758)
    if fp8:
        k[first, 0, 5, 0] = 2.25
        scales = np.ones((c.NB, 1, 2), np.float32)
        codes = np.stack([ow.nearest_e4m3(k), ow.nearest_e4m3(v)], 2)
        c.cache, c.values = (dev(codes), dev(scales)), ow.e4m3_values(codes)
    else:
        kv = [k.astype(np.float16), v.astype(np.float16)]
        c.cache, c.values = tuple(dev(x) for x in kv), np.stack(kv, 2).astype(np.float64)
    out = c.out()
    c.run(1.0, out)
    check(out, c.reference(1.0), 8 * 2.25, 1.0, 0, D)


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_of_any_size_and_minus_infinity(fp8):
    """Finite scores of up to 2^38 (the largest ones' rows come out), rows all of whose scores are minus infinity (0)."""
    D, n = 64, 200
    c = Case([n, n], (4, 1, D), 0 if fp8 else 1000, 0, fp8, seed=11)
    c.q = (c.q * 1000).astype(np.float16)
    if fp8:
        c.scales[:, :, 0] = 2.0 ** 7
        c.values = ow.e4m3_values(c.codes) * c.scales.astype(np.float64)[..., None, None]
        c.cache = c.cache[0], dev(c.scales)
    else:
        k = np.round(c.values[:, :, 0] * 8000)
        c.values[:, :, 0] = k
        c.cache = dev(k.astype(np.float16)), dev(np.nan_to_num(c.values[:, :, 1]).astype(np.float16))
        c.values = np.nan_to_num(c.values)
    out = c.out()
    for scale in (1.0, 50.0, -50.0):
        c.run(scale, out)
        got, s = out.cpu().numpy(), None
        assert np.isfinite(got).all()
        for b in range(2):
            k, v = c.rows(b, np.arange(n))
            for h in range(4):
                s = k[:, 0] @ c.q[b, h].astype(np.float64) * scale
                near = np.sort(s)[-2:]
                if near[1] - near[0] > 2 ** 14 * abs(scale):  # one row has it all, past any rounding of the scores
                    np.testing.assert_allclose(got[b, h], v[s.argmax(), 0], rtol=2.0 ** -10, atol=1e-9)


def test_minus_infinite_keys():
    D = 64
    for window, n in ((20, 100), (1000, 40)):
        c = Case([n], (4, 1, D), window, 0, False, seed=12)
        c.q[:] = 1
        k, v = c.cache[0].cpu().numpy(), np.nan_to_num(c.cache[1].cpu().numpy(), nan=0, posinf=0, neginf=0)
        k[:] = -np.inf
        c.cache = dev(k), dev(v)
        out = c.out()
        c.run(1.0, out)
        assert (out == 0).all()
        last = c.table[0, (n - 1) // BS], 0, (n - 1) % BS
        k[last] = 0
        c.cache = dev(k), dev(v)
        c.run(1.0, out)
        np.testing.assert_allclose(out.cpu().numpy()[0], np.tile(v[last], (4, 1)), rtol=1e-6)


@pytest.mark.parametrize("ctx", [[300, 20], [30000]])
def test_a_visible_nan_is_in_the_output(ctx):
    """Whichever CTA or part of the context has it; the other heads' and sequences' rows are as they were."""
    for fp8 in (False, True):
        c = Case(ctx, (4, 2, 64), 0 if fp8 else 2 ** 20, 0, fp8, seed=13)
        want = c.out()
        c.run(0.125, want)
        for p in (0, ctx[0] // 2, ctx[0] - 1):
            bad = [x.clone() for x in c.cache]
            blk = int(c.table[0, p // BS])
            if fp8:
                bad[0][blk, 1, 0, p % BS, 3] = 0x7f
            else:
                bad[0][blk, 1, p % BS, 3] = float("nan")
            keep, c.cache = c.cache, tuple(bad)
            out = c.out()
            c.run(0.125, out)
            c.cache = keep
            assert out[0, 2:].isnan().all()
            assert torch.equal(out[0, :2], want[0, :2]) and torch.equal(out[1:], want[1:])


@pytest.mark.parametrize("heads", [(14, 2, 64), (32, 8, 128), (20, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (40, 33), (1000, 0)])
def test_fused_append_is_append_then_attention(heads, window, sinks):
    Hq, Hkv, D = heads
    c = Case(CTX, heads, window, sinks, False, seed=21)
    rng = np.random.default_rng(22)
    new = [dev(rng.standard_normal((len(CTX), Hkv, D)).astype(np.float16)) for _ in range(2)]
    before = [x.clone() for x in c.cache]
    out = c.out()
    c.run(0.125, out, k_new=new[0], v_new=new[1])
    fused = [x.clone() for x in c.cache]
    for x, y in zip(c.cache, before):
        x.copy_(y)
    for b, n in enumerate(CTX):
        for x, y in zip(c.cache, new):
            x[int(c.table[b, (n - 1) // BS]), :, (n - 1) % BS] = y[b]
    for x, y in zip(c.cache, fused):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    again = c.out()
    c.run(0.125, again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_lengths_and_blocks_are_flagged(fp8):
    """A length out of range: zeros; a block out of range: left out.  The other sequences are as they were."""
    c = Case([100, 100, 50, 60], (4, 2, 64), 60, 4, fp8, seed=31)
    want = c.out()
    c.run(0.125, want, most=100)
    for bad in (0, -5, 101, 2 ** 31 - 1):
        keep, c.ctx = c.ctx, np.array([100, bad, 50, 60], np.int32)
        out = c.out()
        c.run(0.125, out, most=100)
        c.ctx = keep
        assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["CONTEXT"]
        assert (out[1] == 0).all() and torch.equal(out[[0, 2, 3]], want[[0, 2, 3]])
    for bad in (-1, c.NB, 2 ** 31 - 1):
        keep, c.table = c.table, c.table.copy()
        c.table[1, 4] = bad
        out = c.out()
        c.run(0.125, out, most=100)
        c.table = keep
        assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["BLOCK_ID"]
        assert torch.equal(out[[0, 2, 3]], want[[0, 2, 3]])
        p = ow.visible(100, 60, 4)
        p = p[p // BS != 4]
        k, v = c.rows(1, p)
        for h in range(4):
            np.testing.assert_allclose(out[1, h].cpu().numpy(), ow.attend(c.q[1, h], k[:, h // 2], v[:, h // 2], 0.125), atol=1e-4)


@pytest.mark.parametrize("fp8", [False, True])
def test_checked_mode_refuses_what_a_query_would_see(fp8):
    c = Case([100, 100], (4, 2, 64), 60, 4, fp8, seed=32)
    kvc.kvc_set_checked_mode(True)
    try:
        c.run(0.125, c.out(), most=100)  # entries of blocks in which nothing is visible are out of range
        for change, name in ((dict(ctx=[100, 0]), "KVC_ERR_CAPACITY"), (dict(ctx=[101, 5]), "KVC_ERR_CAPACITY")):
            keep, c.ctx = c.ctx, np.array(change["ctx"], np.int32)
            with pytest.raises(kvc.KvcError) as e:
                c.run(0.125, c.out(), most=100)
            assert e.value.name == name
            c.ctx = keep
        c.table[1, 5] = -1
        with pytest.raises(kvc.KvcError) as e:
            c.run(0.125, c.out(), most=100)
        assert e.value.name == "KVC_ERR_INVALID"
    finally:
        kvc.kvc_set_checked_mode(False)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("overlap", [False, True])
def test_prepared_captured_and_on_another_stream(fp8, overlap):
    cases = [Case([300, 17, 30000], (4, 2, 64), w, 4 if w else 0, fp8, seed=40 + w) for w in ((0, 100) if fp8 else (100, 9000))]
    want = [c.out() for c in cases]
    for c, w in zip(cases, want):
        c.run(0.125, w)
    kvc.kvc_set_launch_overlap(overlap)
    try:
        outs = [c.out() for c in cases]
        calls = [c.run(0.125, o, prepare=True) for c, o in zip(cases, outs)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for call in calls:
            call(side)
        side.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
            o.fill_(float("nan"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for call in calls:
                call()
        for _ in range(3):
            g.replay()
            torch.cuda.synchronize()
            for o, w in zip(outs, want):
                assert torch.equal(o, w)
                o.fill_(float("nan"))
    finally:
        kvc.kvc_set_launch_overlap(False)


def test_offsets_beyond_32_bits():
    """Blocks at the end of pools of more than 2^32 bytes."""
    for fp8 in (False, True):
        Hkv, D, NB = 8, 128, 140000
        shape = (NB, Hkv, 2, BS, D) if fp8 else (NB, Hkv, BS, D)
        c = Case([100, 33], (8, Hkv, D), 90, 5, fp8, seed=51)
        ref = c.reference(0.1)
        top, vmax = c.limits(0.1)
        if fp8:
            big = torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda"), torch.zeros(NB, Hkv, 2, device="cuda")
        else:
            big = tuple(torch.full(shape, float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
        for x, y in zip(big, c.cache):
            x[-c.NB:] = y
        c.cache = big
        ok = (c.table >= 0) & (c.table < c.NB)
        c.table[ok] += NB - c.NB
        out = c.out()
        c.run(0.1, out)
        check(out, ref, top, vmax, 100, D)
        del big, c
        torch.cuda.empty_cache()


@pytest.mark.parametrize("fp8", [False, True])
def test_largest_batch_and_group(fp8):
    """65,535 sequences of one or two tokens in the same blocks; 64 query heads to a KV head."""
    B, D = 65535, 64
    rng = np.random.default_rng(61)
    if fp8:
        codes = rng.integers(0, 0x7e, (4, 1, 2, BS, D)).astype(np.uint8)
        cache = dev(codes), torch.ones(4, 1, 2, device="cuda")
        v = ow.e4m3_values(codes[:, 0, 1])
    else:
        kv = rng.standard_normal((2, 4, 1, BS, D)).astype(np.float16)
        cache, v = (dev(kv[0]), dev(kv[1])), kv[1, :, 0].astype(np.float64)
    table = rng.integers(0, 4, (B, 1)).astype(np.int32)
    ctx = rng.integers(1, 3, B).astype(np.int32)
    q, out = torch.zeros(B, 1, D, dtype=torch.float16, device="cuda"), torch.full((B, 1, D), 9.0, device="cuda")
    args = (q, *cache, dev(table), dev(ctx))
    if fp8:
        assert kvc.paged_decode_fp8_block_plan(B, 1, 1, D, 16) == 0
        kvc.paged_decode_attention_fp8_block(*args, 1.0, out, None, 16)
    else:
        assert kvc.paged_decode_window_plan(B, 1, 1, D, 16, 1) == 0
        kvc.paged_decode_window_attention(*args, 1, 0, 1.0, out, None, 16)
    t, n = table[:, 0], ctx[:, None]
    want = np.where(n == 1, v[t, 0], (v[t, 0] + v[t, 1]) / 2 if fp8 else v[t, 1])
    np.testing.assert_allclose(out[:, 0].cpu().numpy(), want, rtol=1e-6, atol=1e-6)
    c = Case([100, 1, 33], (64, 1, 128), 40, 3, fp8, seed=62)
    top, vmax = c.limits(0.1)
    out = c.out()
    c.run(0.1, out)
    check(out, c.reference(0.1), top, vmax, 100, 128)
    assert kvc.kvc_device_error_flags(clear=True) == 0


def test_scales_that_no_append_writes():
    """Scales of zero and of any positive value are taken as they are."""
    c = Case([150, 40], (4, 2, 64), 0, 0, True, seed=63)
    rng = np.random.default_rng(63)
    scales = rng.uniform(0.001, 0.02, c.scales.shape).astype(np.float32)
    scales[rng.random(scales.shape) < 0.2] = 0
    c.values = ow.e4m3_values(c.codes) * scales.astype(np.float64)[..., None, None]
    c.cache = c.cache[0], dev(np.where(np.isnan(c.cache[1].cpu().numpy()), np.nan, scales).astype(np.float32))
    top, vmax = c.limits(0.3)
    out = c.out()
    c.run(0.3, out)
    # (a scale that is no power of two: its product with the reference's reciprocal, and a rescaled accumulator, are
    # rounded, 2^-24 each and at most once a pair of blocks)
    check(out, c.reference(0.3), top, vmax, 150, 64, 2.0 ** -18)


# ---------------------------------------------------------------- the block-scaled append
def runs(lens, firsts, rng, blocks, skip=()):
    """Slots of runs of tokens, each from an offset `first` of a block of its own on; -1 between some."""
    slots = []
    ids = list(rng.permutation(blocks))
    for n, first in zip(lens, firsts):
        pos, blk = first, None
        for i in range(n):
            if blk is None or pos % BS == 0:
                blk = ids.pop()
            slots.append(blk * BS + pos % BS)
            pos += 1
        if n in skip:
            slots += [-1, -9]
    return np.array(slots, np.int64)


@pytest.mark.parametrize("Hkv,D", [(2, 64), (8, 128), (3, 64), (1, 128)])
@pytest.mark.parametrize("lens,firsts", [
    ([1], [0]), ([1], [15]), ([16], [0]), ([17], [3]), ([1] * 37, list(range(16)) + list(range(16)) + [0] * 5),
    ([5, 1, 40, 33, 2, 16, 100, 7], [11, 0, 15, 0, 14, 1, 9, 4]), ([1500, 3, 700], [7, 13, 0]), ([1] * 5000, [6, 0, 15, 3] * 1250)])
def test_append_fp8_block(Hkv, D, lens, firsts):
    rng = np.random.default_rng(sum(lens) + Hkv)
    blocks = sum(-(-(n + f) // BS) for n, f in zip(lens, firsts)) + 2
    slots = runs(lens, firsts, rng, blocks, skip=(5, 33, 3))
    n = len(slots)
    size = 2.0 ** rng.integers(-6, 7, (n, Hkv, 1))
    k, v = ((rng.standard_normal((n, Hkv, D)) * size).astype(np.float16) for _ in range(2))
    k[rng.random(n) < 0.1] = 0
    codes = rng.integers(0, 256, (blocks, Hkv, 2, BS, D)).astype(np.uint8)
    scales = (2.0 ** rng.integers(-14, 2, (blocks, Hkv, 2))).astype(np.float32)
    got = dev(codes), dev(scales)
    rows = torch.cat((dev(k), dev(v)), 1)  # the tokens apart, as in one projection's output
    if n == 1:
        rows = rows.expand(2, -1, -1).contiguous()[:1]
    kvc.kv_append_fp8_block(rows[:, :Hkv], rows[:, Hkv:], dev(slots), *got)
    ow.append(k, v, slots, codes, scales)
    np.testing.assert_array_equal(got[1].cpu().numpy(), scales)
    g = got[0].cpu().numpy()
    nan = (codes & 0x7f) == 0x7f
    np.testing.assert_array_equal(g[~nan], codes[~nan])
    assert ((g[nan] & 0x7f) == 0x7f).all()
    assert kvc.kvc_device_error_flags(clear=True) == 0


@pytest.mark.parametrize("D", [64, 128])
def test_append_fp8_block_of_long_prompts(D):
    """Prompts of thousands of tokens and many heads: 16 tokens to a warp, runs that end inside its tokens and past them."""
    test_append_fp8_block(8, D, [6001, 3, 700, 1, 90], [7, 13, 0, 4, 15])


def test_append_fp8_block_edges():
    """Largest and smallest values, ties, infinities and NaN, float8 tensors, slots out of range."""
    D = 64
    special = [65504, 57344, 57345, 61440, 448, 449, 464, 2.0 ** -24, 2.0 ** -14, 1.75, 1.7509765625, 0.0]
    for x in special + [np.inf, np.nan]:
        k = np.zeros((2, 1, D), np.float16)
        k[0, 0, :4] = [x, -x, x / 2, 1 / 3 if x < 100 else 100]
        k[1, 0, :2] = [np.inf, x] if np.isfinite(x) else [1.0, -0.5]
        v = -k[:, :, ::-1]
        codes, scales = np.zeros((3, 1, 2, BS, D), np.uint8), np.zeros((3, 1, 2), np.float32)
        got = dev(codes).view(torch.float8_e4m3fn), dev(scales)
        slots = np.array([20, 21], np.int64)
        scales[1] = 2.0 ** -32
        got[1][1] = 2.0 ** -32
        kvc.kv_append_fp8_block(dev(k), dev(v), dev(slots), *got)
        ow.append(k, v, slots, codes, scales)
        np.testing.assert_array_equal(got[1].cpu().numpy(), scales)
        np.testing.assert_array_equal(got[0].float().cpu().numpy(), ow.e4m3_values(codes).astype(np.float32))
    codes, scales = torch.zeros(3, 1, 2, BS, D, dtype=torch.uint8, device="cuda"), torch.zeros(3, 1, 2, device="cuda")
    kvc.kv_append_fp8_block(dev(k), dev(v), dev(np.array([48, 2 ** 40], np.int64)), codes, scales)
    assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["SLOT"]
    assert (codes == 0).all() and (scales == 0).all()
    kvc.kvc_set_checked_mode(True)
    try:
        for slots, name in (([48, 0], "KVC_ERR_CAPACITY"), ([0, 0], "KVC_ERR_INVALID"), ([1, 0], "KVC_ERR_INVALID"),
                            ([1, 3], "KVC_ERR_INVALID")):
            with pytest.raises(kvc.KvcError) as e:
                kvc.kv_append_fp8_block(dev(k), dev(v), dev(np.array(slots, np.int64)), codes, scales)
            assert e.value.name == name
        kvc.kv_append_fp8_block(dev(k), dev(v), dev(np.array([15, 16], np.int64)), codes, scales)
    finally:
        kvc.kvc_set_checked_mode(False)


# ---------------------------------------------------------------- tables
def tables(before, after, free, placed, table, window, sinks, num_slots, positions=True, **kw):
    B = len(after)
    got = [dev(np.asarray(table, np.int32)), torch.full((1,), -77, dtype=torch.int32, device="cuda"),
           torch.full((B + 1,), -77, dtype=torch.int32, device="cuda"),
           torch.full((num_slots,), -77, dtype=torch.int64, device="cuda"),
           torch.full((num_slots,), -77, dtype=torch.int32, device="cuda") if positions else None]
    kvc.kv_block_tables(None if before is None else dev(np.asarray(before, np.int32)), dev(np.asarray(after, np.int32)),
                        dev(np.asarray(free, np.int32)), dev(np.array([placed], np.int32)), *got, window=window, sinks=sinks, **kw)
    return got


def same(got, want):
    for g, w in zip(got, want):
        if g is not None:
            np.testing.assert_array_equal(g.cpu().numpy().ravel(), np.ravel(w))


@pytest.mark.parametrize("B", [1, 2, 5, 31, 511, 512, 513, 1025, 3000])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (16, 4), (33, 20), (1000, 0)])
def test_tables(B, window, sinks):
    rng = np.random.default_rng(B + window)
    most = 600 if B < 40 else 60
    free = rng.permutation(B * 42 + 50).astype(np.int32)
    table, placed, lens = np.full((B, most // BS + 3), -3, np.int32), 3, np.zeros(B, np.int64)
    for step in range(4):
        after = lens + (rng.integers(0, most, B) if step == 0 else rng.integers(0, 2, B))
        n = int((after - lens).sum()) + int(rng.integers(0, 40))
        want = ow.block_tables(lens if step else None, after, free, placed, table, window, sinks, n)
        same(tables(lens if step else None, after, free, placed, table, window, sinks, n, positions=step != 1), want)
        table, placed, lens = want[0], want[1], after
    assert kvc.kvc_device_error_flags(clear=True) == 0


def test_tables_of_long_prompts_and_many_sequences():
    for after, window, sinks in (([200000, 1, 0, 77777], 0, 0), ([200000, 1, 0, 77777], 4096, 4), ([1] * 65535, 0, 0),
                                 ([0] * 65534 + [1000], 16, 0)):
        after = np.array(after)
        free = np.random.default_rng(1).permutation(70000 + sum(-(-after // BS))).astype(np.int32)
        table = np.full((len(after), -(-max(after) // BS)), -1, np.int32)
        n = int(after.sum()) + 5
        same(tables(None, after, free, 0, table, window, sinks, n), ow.block_tables(None, after, free, 0, table, window, sinks, n))
    assert kvc.kvc_device_error_flags(clear=True) == 0


def test_tables_are_all_or_nothing():
    free, table = np.arange(10, 16, dtype=np.int32), np.arange(12, dtype=np.int32).reshape(2, 6)
    for before, after, placed, n in (([0, 0], [64, 33], 0, 97), ([16, 0], [17, 64], 2, 99), ([0, 0], [16, 16], 0, 31),
                                     ([5, 5], [6, 6], -1, 9), ([5, 5], [6, 6], 7, 9), ([0, 0], [90, 96], 0, 0)):
        want = (table, placed, np.zeros(3), np.full(n, -1), np.zeros(n))
        same(tables(before, after, free, placed, table, 0, 0, n), want)
        assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["BLOCKS"]
    # exactly enough
    same(tables([0, 0], [64, 32], free, 0, table, 0, 0, 96), ow.block_tables([0, 0], [64, 32], free, 0, table, 0, 0, 96))
    same(tables([5, 5], [6, 6], free, 6, table, 0, 0, 2), ow.block_tables([5, 5], [6, 6], free, 6, table, 0, 0, 2))
    assert kvc.kvc_device_error_flags(clear=True) == 0
    # lengths that do not fit: that sequence gets nothing
    for lo, hi in ((-1, 5), (6, 5), (0, 97), (0, 2 ** 31 - 1), (-2 ** 31, 2 ** 31 - 1)):
        want = ow.block_tables([lo, 17], [hi, 40], free, 1, table, 0, 0, 30)
        same(tables([lo, 17], [hi, 40], free, 1, table, 0, 0, 30), want)
        assert kvc.kvc_device_error_flags(clear=True) == kvc.DEVERR["CONTEXT"]
        kvc.kvc_set_checked_mode(True)
        try:
            with pytest.raises(kvc.KvcError):
                tables([lo, 17], [hi, 40], free, 1, table, 0, 0, 30)
            with pytest.raises(kvc.KvcError, match="blocks"):
                tables([0, 17], [96, 40], free, 1, table, 0, 0, 200)
            with pytest.raises(kvc.KvcError, match="tokens"):
                tables([0, 17], [1, 40], free, 1, table, 0, 0, 20)
            same(tables([3, 17], [4, 40], free, 1, table, 0, 0, 30), ow.block_tables([3, 17], [4, 40], free, 1, table, 0, 0, 30))
        finally:
            kvc.kvc_set_checked_mode(False)
    # no sequences, no room, no blocks
    same(tables([0], [0], np.zeros(0, np.int32), 0, table[:1], 0, 0, 0), (table[:1], 0, [0, 0], [], []))
    same(tables(np.zeros(0), np.zeros(0), free, 2, table[:0], 0, 0, 3), (table[:0], 2, [0], [-1] * 3, [0] * 3))
    assert kvc.kvc_device_error_flags(clear=True) == 0


# ---------------------------------------------------------------- prefill
def packed(lens, heads, seed):
    rng = np.random.default_rng(seed)
    Hq, Hkv, D = heads
    q, k, v = (rng.standard_normal((sum(lens), h, D)).astype(np.float16) for h in (Hq, Hkv, Hkv))
    return q, k, v, np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def prefill_reference(q, k, v, lens, scale, window, sinks):
    """The oracle's definition, a segment at a time in torch's 64 bits (on the GPU: the long cases)."""
    q, k, v = (dev(x).double() for x in (q, k, v))
    out, at, per = torch.zeros_like(q), 0, q.shape[1] // k.shape[1]
    for n in lens:
        i, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
        hidden = ~((j <= i) & ((j > i - window) | (j < sinks)))
        for h in range(q.shape[1]):
            s = (q[at:at + n, h] @ k[at:at + n, h // per].T * scale).masked_fill(hidden, -np.inf)
            out[at:at + n, h] = torch.softmax(s, -1) @ v[at:at + n, h // per]
        at += n
    return out.cpu().numpy()


def run_prefill(q, k, v, cu, scale, window, sinks, dtype, precise=False, **kw):
    out = torch.full(q.shape, float("nan"), dtype=dtype, device="cuda")
    kvc.prefill_window_attention(dev(q), dev(k), dev(v), dev(cu), int(np.diff(cu).max()), window, sinks, scale, out,
                                 precise=precise, **kw)
    return out


def check_prefill(out, ref, q, k, v, scale, n, precise):
    D = q.shape[2]
    top = float(np.abs(q.astype(np.float64)).max(0).max(0) @ np.abs(k.astype(np.float64)).max(0).max(0)) * abs(scale)
    # fp16 weights: 2^-11 each, and those below 2^-25 of the largest are lost; the split form keeps 2^-20
    extra = n * 2.0 ** -25 + (0 if precise else 2.0 ** -11)
    check(out, ref, min(top, 40.0), float(np.abs(v.astype(np.float64)).max()), n, D, extra)


@pytest.mark.parametrize("heads", [(4, 2, 64), (4, 1, 128), (14, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 4), (127, 0), (128, 128), (129, 130), (200, 300), (256, 16),
                                          (384, 1), (1000, 4), (40, 1000)])
def test_prefill_windows(heads, window, sinks):
    lens = [1, 700, 128, 0, 129, 37, 512, 385]
    q, k, v, cu = packed(lens, heads, window)
    scale = heads[2] ** -0.5
    ref = prefill_reference(q, k, v, lens, scale, window, sinks)
    for dtype, precise in ((torch.float16, False), (torch.float32, True), (torch.float32, False)):
        out = run_prefill(q, k, v, cu, scale, window, sinks, dtype, precise)
        check_prefill(out, ref, q, k, v, scale, 700, precise)
    assert kvc.kvc_device_error_flags(clear=True) == 0


@pytest.mark.parametrize("heads,lens,window,sinks", [((16, 4, 64), [4097, 511], 300, 4), ((16, 4, 64), [4200], 1111, 140),
                                                     ((4, 2, 128), [3333, 1], 700, 260), ((16, 2, 64), [256 * 18], 1, 0)])
@pytest.mark.parametrize("scale", [0.125, -0.3, 0.0])
def test_prefill_of_long_prompts(heads, lens, window, sinks, scale):
    """Also at head dim 64 with two query tiles to a CTA."""
    q, k, v, cu = packed(lens, heads, 7)
    ref = prefill_reference(q, k, v, lens, scale, window, sinks)
    out = run_prefill(q, k, v, cu, scale, window, sinks, torch.float32)
    check_prefill(out, ref, q, k, v, scale, window + sinks, False)
    assert kvc.kvc_device_error_flags(clear=True) == 0


@pytest.mark.parametrize("nseq", [255, 256, 257, 700])
@pytest.mark.parametrize("heads", [(2, 1, 64), (3, 3, 128)])
def test_prefill_of_many_prompts(nseq, heads):
    """Listed segments (up to 256) and more than that; empty ones among them."""
    lens = list(np.random.default_rng(nseq).integers(0, 40, nseq))
    lens[3], lens[nseq - 2], lens[nseq - 1] = 300, 600, 0
    q, k, v, cu = packed(lens, heads, 13)
    ref = prefill_reference(q, k, v, lens, 0.2, 33, 5)
    check_prefill(run_prefill(q, k, v, cu, 0.2, 33, 5, torch.float32), ref, q, k, v, 0.2, 40, False)
    assert kvc.kvc_device_error_flags(clear=True) == 0


def test_prefill_reference_is_the_oracles():
    lens = [9, 40]
    q, k, v, cu = packed(lens, (4, 2, 64), 8)
    np.testing.assert_allclose(prefill_reference(q, k, v, lens, 0.2, 7, 3), ow.prefill(q, k, v, lens, 0.2, 7, 3), atol=1e-12)


@pytest.mark.parametrize("heads", [(2, 1, 64), (2, 1, 128), (64, 1, 64)])
def test_prefill_hidden_infinities_and_nan(heads):
    """Rows that do not see a position are finite and the definition's whatever it holds; rows that see it have it.

    (A row in whose tiles such a value lay is computed again, its weights in fp32 instead of fp16: either result is within
    check_prefill's bound of the definition, 2^-11 a weight, but they need not be the same bits.)"""
    lens, window, sinks, scale = [700, 400], 150, 3, 0.125
    q, k, v, cu = packed(lens, heads, 9)
    ref = prefill_reference(q, k, v, lens, scale, window, sinks)
    for precise in (False, True):
        clean = run_prefill(q, k, v, cu, scale, window, sinks, torch.float32, precise)
        for p in (0, 2, 3, 127, 300, 699, 700, 1099):
            for value in (np.inf, np.nan):
                for which in range(2):
                    kv = [k.copy(), v.copy()]
                    kv[which][p, 0, 5] = value
                    out = run_prefill(q, *kv, cu, scale, window, sinks, torch.float32, precise)
                    seg0, n = (0, 700) if p < 700 else (700, 400)
                    i = np.arange(n)
                    sees = (p - seg0 <= i) & ((p - seg0 > i - window) | (p - seg0 < sinks))
                    rows = np.zeros(1100, bool)
                    rows[seg0:seg0 + n] = sees
                    got, want = out.cpu().numpy(), clean.cpu().numpy()
                    check_prefill(out[dev(~rows)], ref[~rows], q, k, v, scale, 700, precise)
                    if which == 1:
                        assert not np.isfinite(got[rows][:, :, 5]).any()
                        other = np.arange(heads[2]) != 5
                        np.testing.assert_allclose(got[rows][:, :, other], want[rows][:, :, other], atol=4e-3)
                    elif np.isnan(value):
                        assert np.isnan(got[rows]).all()
    assert kvc.kvc_device_error_flags(clear=True) == 0


def test_prefill_rows_of_minus_infinity_are_zero():
    lens = [200]
    q, k, v, cu = packed(lens, (2, 1, 64), 10)
    q[:] = 1
    k[50:120] = -np.inf
    out = run_prefill(q, k, v, cu, 0.125, 20, 0, torch.float32).cpu().numpy()
    assert (out[50 + 19:120] == 0).all() and np.isfinite(out).all()
    ref = prefill_reference(q, np.where(np.isinf(k), 0, k).astype(np.float16), v, lens, 0.125, 20, 0)
    np.testing.assert_allclose(out[:50], ref[:50], atol=4e-3)


def test_prefill_bad_segments_are_flagged():
    q, k, v, cu = packed([60, 40], (2, 1, 64), 11)
    want = run_prefill(q, k, v, cu, 0.125, 20, 0, torch.float32)
    for bad in ([0, 60, 101], [0, -1, 100], [0, 120, 100]):
        out = torch.full(q.shape, 7.0, device="cuda")
        kvc.prefill_window_attention(dev(q), dev(k), dev(v), dev(np.array(bad, np.int32)), 60, 20, 0, 0.125, out)
        assert kvc.kvc_device_error_flags(clear=True) & kvc.DEVERR["SEQLENS"]
        if bad[1] == 60:
            assert torch.equal(out[:60], want[:60])
    kvc.kvc_set_checked_mode(True)
    try:
        with pytest.raises(kvc.KvcError):
            kvc.prefill_window_attention(dev(q), dev(k), dev(v), dev(np.array([0, 60, 90], np.int32)), 60, 20, 0, 0.125, want)
    finally:
        kvc.kvc_set_checked_mode(False)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_outputs_aligned_to_16_bytes(D, dtype):
    """An output that begins 16 bytes behind a 32-byte boundary, or on one: the same values, nothing beside them."""
    q, k, v, cu = packed([60, 300], (2, 1, D), 14)
    want = run_prefill(q, k, v, cu, 0.125, 20, 2, dtype)
    step = 16 // want.element_size()
    for shift in (0, step, 2 * step, 3 * step):
        room = torch.full((want.numel() + 4 * step,), 5.0, dtype=dtype, device="cuda")
        out = room[shift:shift + want.numel()].view(want.shape)
        kvc.prefill_window_attention(dev(q), dev(k), dev(v), dev(cu), 300, 20, 2, 0.125, out)
        assert torch.equal(out, want)
        assert (room[:shift] == 5).all() and (room[shift + want.numel():] == 5).all()
    assert kvc.kvc_device_error_flags(clear=True) == 0


def test_prefill_of_any_max_seqlen():
    """max_seqlen may be as large as its type: no segment is longer than all tokens."""
    q, k, v, cu = packed([60, 300], (2, 1, 64), 13)
    want = run_prefill(q, k, v, cu, 0.125, 20, 2, torch.float32)
    for most in (2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30):
        out = torch.zeros_like(want)
        kvc.prefill_window_attention(dev(q), dev(k), dev(v), dev(cu), most, 20, 2, 0.125, out)
        assert torch.equal(out, want)
    assert kvc.kvc_device_error_flags(clear=True) == 0


def test_prefill_captured_behind_the_tables():
    """cu_tokens of kv_block_tables are prefill's cu_seqlens; both captured into one graph."""
    lens = [130, 1, 260]
    q, k, v, cu = packed(lens, (4, 2, 64), 12)
    want = run_prefill(q, k, v, cu, 0.125, 50, 4, torch.float16)
    after, free = dev(np.array(lens, np.int32)), dev(np.arange(90, dtype=np.int32))
    placed, new_placed, got_cu = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, 1, 4))
    table, slots = torch.zeros(3, 17, dtype=torch.int32, device="cuda"), torch.zeros(391, dtype=torch.int64, device="cuda")
    out = torch.zeros_like(want)
    tensors = [dev(x) for x in (q, k, v)]
    calls = (kvc.kv_block_tables(None, after, free, placed, table, new_placed, got_cu, slots, prepare=True),
             kvc.prefill_window_attention(*tensors, got_cu, 260, 50, 4, 0.125, out, prepare=True))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in calls:
            call()
    for _ in range(2):
        got_cu.zero_()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# ---------------------------------------------------------------- all of them together
@pytest.mark.parametrize("block8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3), (33, 40)])
@pytest.mark.parametrize("heads", [(14, 2, 64), (8, 2, 128)])
def test_serving_prompts_and_steps(block8, window, sinks, heads):
    """Prompts, then a captured step replayed 60 times: tables, cache contents and attention as the definitions have them,
    step by step; a windowed sequence's blocks come round, and no more are taken."""
    from paged_kv_cache_27_gb300.harness import ServingSession
    Hq, Hkv, D = heads
    lens, steps = [1, 70, 16, 47], 60
    B, NB, most = len(lens), 64, 144
    s = ServingSession(B, Hq, Hkv, D, NB, most, window, sinks, block8, out_dtype=torch.float32)
    rng = np.random.default_rng(window + D)
    free = s.free.cpu().numpy()
    table, placed, before = np.full((B, most // BS), -1, np.int32), 0, None
    codes, scales = np.full((NB, Hkv, 2, BS, D), 0x7f, np.uint8), np.full((NB, Hkv, 2), np.nan)
    kv = np.full((NB, Hkv, 2, BS, D), np.nan)

    def placed_rows(after, k, v):
        nonlocal table, placed, before
        table, placed, _, slots, _ = ow.block_tables(before, after, free, placed, table, window, sinks, len(k))
        before = np.array(after)
        if block8:
            ow.append(k, v, slots, codes, scales)
        for t, slot in enumerate(slots):
            if slot >= 0:
                kv[slot // BS, :, 0, slot % BS], kv[slot // BS, :, 1, slot % BS] = k[t], v[t]

    def values(b, p):
        x = kv if not block8 else ow.e4m3_values(codes) * scales[..., None, None]
        x = x[table[b, p // BS], :, :, p % BS]
        return x[:, :, 0], x[:, :, 1]

    q, k, v, cu = packed(lens, heads, 31)
    got = s.prompts(dev(q), dev(k), dev(v), lens)
    ref = prefill_reference(q, k, v, lens, s.scale, window or 10 ** 6, sinks)
    check_prefill(got, ref, q, k, v, s.scale, 100, False)
    placed_rows(lens, k, v)
    s.step()  # (a warm-up whose token stays)
    zeros = [np.zeros((B, h, D), np.float16) for h in (Hkv, Hkv)]
    placed_rows(before + 1, *zeros)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.step()
    for step in range(steps):
        q, k, v = (rng.standard_normal((B, h, D)).astype(np.float16) for h in (Hq, Hkv, Hkv))
        for t, a in ((s.q, q), (s.k, k), (s.v, v)):
            t.copy_(dev(a))
        g.replay()
        placed_rows(before + 1, k, v)
        if step % 7 and step != steps - 1:
            continue
        np.testing.assert_array_equal(s.table.cpu().numpy(), table)
        assert int(s.placed) == placed and np.array_equal(s.before.cpu().numpy(), before)
        if block8:
            used = ~np.isnan(scales)
            np.testing.assert_array_equal(s.scales.cpu().numpy()[used], scales[used])
            np.testing.assert_array_equal(s.codes.cpu().numpy()[used.any((1, 2))], codes[used.any((1, 2))])
        values.ctx = before
        ref = ow.decode(q, values, s.scale, window, sinks)
        top = max(float(np.abs(q[b].astype(np.float64)).max(0) @ np.abs(values(b, ow.visible(int(before[b]), window, sinks))[0])
                        .max((0, 1))) for b in range(B)) * s.scale
        check(s.out, ref, min(top, 40.0), 6.0, most, D)
    if window:
        assert placed <= B * (ow.ring(window) + -(-sinks // BS))
    assert kvc.kvc_device_error_flags(clear=True) == 0
    s.close()


@pytest.mark.parametrize("block8,window", [(False, 0), (False, 50), (True, 0), (True, 50)])
def test_session_with_launch_overlap(block8, window):
    """With launch overlap on, a session's steps read what its tables and appends wrote."""
    from paged_kv_cache_27_gb300.harness import ServingSession
    lens, results = [400, 5, 300], []
    q, k, v, cu = packed(lens, (8, 2, 64), 42)
    try:
        for on in (False, True):
            kvc.kvc_set_launch_overlap(on)
            s = ServingSession(3, 8, 2, 64, 120, 600, window, 4 if window else 0, block8)
            outs = [s.prompts(dev(q), dev(k), dev(v), lens)]
            for i in range(40):
                for t, seed in ((s.q, 1), (s.k, 2), (s.v, 3)):
                    t.copy_(dev(np.random.default_rng([i, seed]).standard_normal(t.shape).astype(np.float16)))
                s.step()
                outs.append(s.out.clone())
            results.append(outs)
            torch.cuda.synchronize()
            s.close()
    finally:
        kvc.kvc_set_launch_overlap(False)
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert kvc.kvc_device_error_flags(clear=True) == 0


def test_two_sessions_on_two_streams():
    """Calls of both at once, each with its own tables, cache and workspace: as one after the other."""
    from paged_kv_cache_27_gb300.harness import ServingSession
    made = []
    for block8, window in ((True, 0), (False, 50)):
        def run(stream):
            with torch.cuda.stream(stream):
                s = ServingSession(3, 8, 2, 64, 200, 900, window, 4 if window else 0, block8)
                q, k, v, cu = packed([800, 5, 300], (8, 2, 64), 41)
                outs = [s.prompts(dev(q), dev(k), dev(v), [800, 5, 300])]
                for i in range(20):
                    for t, seed in ((s.q, 1), (s.k, 2), (s.v, 3)):
                        t.copy_(dev(np.random.default_rng([i, seed]).standard_normal(t.shape).astype(np.float16)))
                    s.step()
                    outs.append(s.out.clone())
            return s, outs
        made.append(run)
    streams = [torch.cuda.Stream() for _ in range(2)]
    alone = []
    for run, st in zip(made, streams):
        alone.append(run(st)[1])
        torch.cuda.synchronize()
    together = [run(st) for run, st in zip(made, streams)]
    torch.cuda.synchronize()
    for a, (_, b) in zip(alone, together):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert kvc.kvc_device_error_flags(clear=True) == 0
