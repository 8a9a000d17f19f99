"""The windowed, block-scaled and table-building oracles against other things than themselves, and the library's
refusals, which need no GPU."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import paged_kv_cache_27_gb300 as kvc
from oracle import window as ow


# ---------------------------------------------------------------- oracles
def test_e4m3_table_and_rounding_are_torchs():
    every = torch.arange(256, dtype=torch.uint8)
    want = every.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ow.e4m3_values(every.numpy()), want)
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(5000) * 2.0 ** rng.integers(-12, 8, 5000), ow.E4M3, -ow.E4M3,
                        (ow.E4M3[1:] + ow.E4M3[:-1]) / 2, [449, 463, -0.0]])
    x = x[np.abs(x) <= 464].astype(np.float32)
    x = x[np.abs(x) <= 448]
    got = ow.nearest_e4m3(x)
    np.testing.assert_array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_exponent_is_the_least():
    rng = np.random.default_rng(2)
    for x in list(rng.standard_normal(200).astype(np.float16) * np.float16(30)) + [np.float16(v) for v in (
            448, 448.25, 449, 65504, 2.0 ** -24, 1.75, 1.7510, 0.875)]:
        e = ow.exponent(np.array([x]))
        assert abs(float(x)) <= 448 * 2.0 ** e
        assert e == ow.LEAST or abs(float(x)) > 448 * 2.0 ** (e - 1)
    assert ow.exponent(np.zeros(4)) == ow.LEAST
    assert ow.exponent(np.array([np.inf, np.nan, 1.0])) == ow.exponent(np.array([1.0]))


def test_a_grown_block_holds_what_appending_at_once_holds_but_for_subnormals():
    rng = np.random.default_rng(3)
    rows = (rng.standard_normal((16, 2, 64)) * 2.0 ** rng.integers(-2, 3, (16, 1, 1))).astype(np.float16)
    at_once, one_by_one = [(np.zeros((1, 2, 2, 16, 64), np.uint8), np.zeros((1, 2, 2))) for _ in range(2)]
    ow.append(rows, rows, np.arange(16), *at_once)
    for t in range(16):
        ow.append(rows[t:t + 1], rows[t:t + 1], np.array([t]), *one_by_one)
    np.testing.assert_array_equal(at_once[1], one_by_one[1])
    a, b = ow.e4m3_values(at_once[0]), ow.e4m3_values(one_by_one[0])
    normal = np.abs(a) >= 2.0 ** -6
    np.testing.assert_array_equal(a[normal], b[normal])
    assert np.abs(a - b).max() <= 2.0 ** -9


def test_window_of_everything_is_causal_attention_and_sinks_come_back():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((9, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    t = [torch.from_numpy(x).transpose(0, 1)[None] for x in (q, k, v)]
    full = torch.nn.functional.scaled_dot_product_attention(*t, is_causal=True, scale=0.3, enable_gqa=True)[0]
    np.testing.assert_allclose(ow.prefill(q, k, v, [9], 0.3, 9, 0), full.transpose(0, 1).numpy(), atol=1e-12)
    np.testing.assert_allclose(ow.prefill(q, k, v, [9], 0.3, 1, 9), full.transpose(0, 1).numpy(), atol=1e-12)
    i, j = np.arange(9)[:, None], np.arange(9)[None]
    mask = torch.from_numpy((j <= i) & ((i - j < 3) | (j < 2)))
    part = torch.nn.functional.scaled_dot_product_attention(*t, attn_mask=mask, scale=0.3, enable_gqa=True)[0]
    np.testing.assert_allclose(ow.prefill(q, k, v, [9], 0.3, 3, 2), part.transpose(0, 1).numpy(), atol=1e-12)


def test_ring_is_the_least_number_of_blocks():
    for window in (1, 2, 15, 16, 17, 18, 31, 32, 33, 1024):
        assert ow.ring(window) == -(-(window + 15) // 16)


def test_tables_of_a_windowed_sequence_keep_what_is_visible():
    """Positions written through the slots, step by step, are there whenever a later query sees them."""
    rng = np.random.default_rng(5)
    for window, sinks in ((1, 0), (5, 3), (16, 16), (17, 20), (40, 4)):
        free = rng.permutation(60).astype(np.int32)
        table, placed, held = np.full((2, 30), -1, np.int32), 0, {}
        lens = np.array([0, 0])
        for new in ((70, 9),) + ((1, 1),) * 150 + ((0, 1),) * 3:
            after = lens + new
            table, placed, cu, slots, pos = ow.block_tables(lens, after, free, placed, table, window, sinks, 90)
            seq = np.searchsorted(cu, np.arange(cu[-1]), side="right") - 1
            for t in range(cu[-1]):
                if slots[t] >= 0:
                    held[int(slots[t])] = (int(seq[t]), int(pos[t]))
            lens = after
            for b in range(2):
                for p in ow.visible(int(lens[b]), window, sinks):
                    assert held[int(table[b, p // 16]) * 16 + p % 16] == (b, p)
        assert placed <= 2 * (ow.ring(window) + -(-sinks // 16))


def test_tables_without_a_window_are_the_host_functions():
    rng = np.random.default_rng(6)
    before, after = np.array([0, 5, 16, 31, 8]), np.array([1, 37, 17, 31, 16])
    table = np.full((5, 6), -1, np.int32)
    ids = rng.permutation(40).astype(np.int32)
    at = 0
    for b in range(5):
        n = -(-before[b] // 16)
        table[b, :n] = ids[at:at + n]
        at += n
    got, placed, cu, slots, pos = ow.block_tables(before, after, ids, at, table, 0, 0, 60)
    want = kvc.kv_slot_mapping(got, before, after - before)
    np.testing.assert_array_equal(slots[:cu[-1]], want)
    np.testing.assert_array_equal(slots[cu[-1]:], -1)
    assert placed == at + sum(-(-after // 16) - -(-before // 16))
    np.testing.assert_array_equal(pos[:cu[-1]], np.concatenate([np.arange(a, b) for a, b in zip(before, after)]))


# ---------------------------------------------------------------- refusals
def at(i, off=0):
    """The i-th of addresses 16 MB apart, more than any buffer below holds."""
    return ctypes.c_void_p((i << 24) + off)


def refused(fn, args, status, text):
    assert kvc.STATUS[getattr(kvc._lib, fn)(*args)] == "KVC_ERR_" + status, (fn, text)
    assert text in kvc._lib.kvc_last_error_string().decode(), (fn, kvc._lib.kvc_last_error_string())


TABLES = dict(before=at(1), after=at(2), B=3, free=at(3), nf=20, placed=at(4), window=0, sinks=0, table=at(5), mb=8, bs=16,
              new=at(6), cu=at(7), slots=at(8), pos=at(9), ns=40, st=None)
APPEND = dict(k=at(1), ks=128, v=at(2), vs=136, n=20, slots=at(3), codes=at(4), scales=at(5), NB=8, Hkv=2, D=64, bs=16,
              st=None)
FP8 = dict(q=at(1), codes=at(2), scales=at(3), NB=8, table=at(4), mb=4, ctx=at(5), window=0, sinks=0, B=2, Hq=4, Hkv=2,
           D=64, bs=16, most=64, scale=0.125, out=at(6), od=0, ws=None, wb=0, st=None)
WINDOW = dict(q=at(1), kn=at(2), vn=at(3), k=at(4), v=at(5), NB=8, table=at(6), mb=4, ctx=at(7), window=20, sinks=4, B=2,
              Hq=4, Hkv=2, D=64, bs=16, most=64, scale=0.125, out=at(8), od=0, ws=None, wb=0, st=None)
PREFILL = dict(q=at(1), k=at(2), v=at(3), cu=at(4), nseq=2, T=30, most=20, Hq=4, Hkv=2, D=64, scale=0.125, window=20,
               sinks=4, prec=0, out=at(5), od=0, st=None)
CALLS = {"kv_block_tables": TABLES, "kv_append_fp8_block": APPEND, "paged_decode_attention_fp8_block": FP8,
         "paged_decode_window_attention": WINDOW, "prefill_window_attention": PREFILL}
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("fn,change,status,text", [
    ("kv_block_tables", dict(B=-1), "INVALID", "sizes"), ("kv_block_tables", dict(mb=0), "INVALID", "sizes"),
    ("kv_block_tables", dict(ns=-1), "INVALID", "sizes"), ("kv_block_tables", dict(B=65536), "UNSUPPORTED", "65535"),
    ("kv_block_tables", dict(bs=32), "UNSUPPORTED", "block_size"),
    ("kv_block_tables", dict(mb=2 ** 27), "UNSUPPORTED", "2^31"),
    ("kv_block_tables", dict(sinks=4), "INVALID", "sinks without"),
    ("kv_block_tables", dict(window=-1), "INVALID", "window"), ("kv_block_tables", dict(window=4, sinks=-1), "INVALID", "sinks"),
    ("kv_block_tables", dict(window=2 ** 30 + 1), "UNSUPPORTED", "window"),
    *[("kv_block_tables", {x: None}, "INVALID", "null") for x in ("after", "free", "placed", "table", "new", "cu", "slots")],
    *[("kv_block_tables", {x: at(12, 2)}, "INVALID", "aligned") for x in ("before", "after", "free", "placed", "table",
                                                                            "new", "cu", "pos")],
    ("kv_block_tables", dict(slots=at(12, 4)), "INVALID", "aligned"),
    *[("kv_block_tables", c, "INVALID", "overlaps") for c in (
        dict(new=at(4)), dict(cu=at(1, 8)), dict(table=at(2, -8)), dict(slots=at(3)), dict(pos=at(8, 316)),
        dict(cu=at(5, 92)), dict(new=at(7, 12)), dict(table=at(3, 76)))],
    ("kv_append_fp8_block", dict(n=-1), "INVALID", "sizes"), ("kv_append_fp8_block", dict(Hkv=0), "INVALID", "sizes"),
    ("kv_append_fp8_block", dict(D=96), "UNSUPPORTED", "head_dim"), ("kv_append_fp8_block", dict(bs=8), "UNSUPPORTED", "block_size"),
    ("kv_append_fp8_block", dict(NB=0), "INVALID", "num_blocks"),
    ("kv_append_fp8_block", dict(NB=2 ** 25), "UNSUPPORTED", "2^30"),
    *[("kv_append_fp8_block", {x: None}, "INVALID", "null") for x in ("k", "v", "slots", "codes", "scales")],
    *[("kv_append_fp8_block", {x: at(12, 8)}, "INVALID", "aligned") for x in ("k", "v", "codes", "scales")],
    ("kv_append_fp8_block", dict(slots=at(12, 4)), "INVALID", "aligned"),
    *[("kv_append_fp8_block", c, "INVALID", "strides") for c in (dict(ks=120), dict(vs=132), dict(ks=0), dict(vs=-128))],
    *[("kv_append_fp8_block", c, "INVALID", "overlaps") for c in (
        dict(codes=at(1)), dict(codes=at(2, 19 * 136 * 2 + 240)), dict(scales=at(3, 144)), dict(scales=at(4, 16)),
        dict(codes=at(5, 112)))],
    ("paged_decode_attention_fp8_block", dict(Hq=5), "INVALID", "multiple"),
    ("paged_decode_attention_fp8_block", dict(D=32), "UNSUPPORTED", "head_dim"),
    ("paged_decode_attention_fp8_block", dict(Hq=130), "UNSUPPORTED", "group"),
    ("paged_decode_attention_fp8_block", dict(B=65536), "UNSUPPORTED", "65535"),
    ("paged_decode_attention_fp8_block", dict(sinks=1), "INVALID", "sinks without"),
    ("paged_decode_attention_fp8_block", dict(window=-1), "INVALID", "window"),
    ("paged_decode_attention_fp8_block", dict(most=65), "CAPACITY", "max_context_len"),
    ("paged_decode_attention_fp8_block", dict(mb=0), "INVALID", "max_blocks"),
    ("paged_decode_attention_fp8_block", dict(mb=2 ** 27), "UNSUPPORTED", "2^31"),
    ("paged_decode_attention_fp8_block", dict(NB=2 ** 25), "UNSUPPORTED", "2^30"),
    ("paged_decode_attention_fp8_block", dict(od=2), "INVALID", "out_dtype"),
    *[("paged_decode_attention_fp8_block", dict(scale=x), "INVALID", "scale") for x in (NAN, INF)],
    *[("paged_decode_attention_fp8_block", {x: None}, "INVALID", "null") for x in ("q", "codes", "scales", "table", "ctx", "out")],
    *[("paged_decode_attention_fp8_block", {x: at(12, 2)}, "INVALID", "aligned") for x in ("q", "codes", "scales", "table",
                                                                                             "ctx", "out")],
    *[("paged_decode_attention_fp8_block", c, "INVALID", "overlaps") for c in (
        dict(out=at(1)), dict(out=at(2, 8 * 2 * 2 * 16 * 64 - 16)), dict(out=at(3, 112)), dict(out=at(4, 16)), dict(out=at(5)))],
    ("paged_decode_window_attention", dict(window=0, sinks=0), "INVALID", "window"),
    ("paged_decode_window_attention", dict(sinks=-1), "INVALID", "sinks"),
    ("paged_decode_window_attention", dict(sinks=2 ** 30 + 1), "UNSUPPORTED", "sinks"),
    ("paged_decode_window_attention", dict(kn=None), "INVALID", "both or neither"),
    ("paged_decode_window_attention", dict(vn=at(12, 8)), "INVALID", "aligned"),
    ("paged_decode_window_attention", dict(NB=0), "INVALID", "num_blocks"),
    ("paged_decode_window_attention", dict(NB=2 ** 26), "UNSUPPORTED", "2^31"),
    ("paged_decode_window_attention", dict(scale=NAN), "INVALID", "scale"),
    *[("paged_decode_window_attention", {x: None}, "INVALID", "null") for x in ("q", "k", "v", "table", "ctx", "out")],
    *[("paged_decode_window_attention", c, "INVALID", "overlaps") for c in (
        dict(out=at(1)), dict(out=at(2)), dict(out=at(4)), dict(k=at(3)), dict(v=at(1, 16)), dict(k=at(6)), dict(v=at(7)),
        dict(k=at(5, 16)), dict(out=at(8), k=at(8, 1008)))],
    ("prefill_window_attention", dict(window=0), "INVALID", "window"), ("prefill_window_attention", dict(sinks=-1), "INVALID", "sinks"),
    ("prefill_window_attention", dict(prec=2), "INVALID", "p_precision"), ("prefill_window_attention", dict(Hq=5), "INVALID", "multiple"),
    ("prefill_window_attention", dict(scale=INF), "INVALID", "scale"), ("prefill_window_attention", dict(D=80), "UNSUPPORTED", "head_dim"),
    ("prefill_window_attention", dict(cu=at(4, 2)), "INVALID", "aligned"), ("prefill_window_attention", dict(v=at(3, 8)), "INVALID", "aligned"),
    *[("prefill_window_attention", {x: None}, "INVALID", "null") for x in ("q", "k", "v", "cu", "out")],
    *[("prefill_window_attention", c, "INVALID", "overlaps") for c in (
        dict(out=at(1)), dict(out=at(2, 30 * 2 * 64 * 2 - 16)), dict(out=at(3)), dict(out=at(4, 0)))],
])
def test_refusals(fn, change, status, text):
    refused(fn, list({**CALLS[fn], **change}.values()), status, text)


def test_empty_calls_are_nothing():
    for fn, change in (("kv_append_fp8_block", dict(n=0, k=None)), ("paged_decode_attention_fp8_block", dict(B=0, q=None)),
                       ("paged_decode_window_attention", dict(B=0, q=None)), ("prefill_window_attention", dict(nseq=0)),
                       ("prefill_window_attention", dict(T=0))):
        assert getattr(kvc._lib, fn)(*{**CALLS[fn], **change}.values()) == 0


def test_plans_refuse_what_the_calls_refuse():
    for bad in (dict(window=-1), dict(sinks=-1), dict(window=0, sinks=1), dict(window=2 ** 30 + 1), dict(head_dim=96),
                dict(Hq=5), dict(max_context_len=0)):
        for fn, least in ((kvc.paged_decode_window_plan, 1), (kvc.paged_decode_fp8_block_plan, 0)):
            with pytest.raises(kvc.KvcError):
                fn(**{**dict(B=2, Hq=4, Hkv=2, head_dim=64, max_context_len=100, window=20, sinks=0), **bad})
    with pytest.raises(kvc.KvcError):
        kvc.paged_decode_window_plan(2, 4, 2, 64, 100, 0)


def test_calls_by_number_are_the_calls():
    call = kvc._lib.kvc_call
    for which, fn in zip(range(16, 21), ("kv_block_tables", "kv_append_fp8_block", "paged_decode_attention_fp8_block",
                                         "paged_decode_window_attention", "prefill_window_attention")):
        n = len(getattr(kvc._lib, fn).argtypes) - 1
        words = struct.pack("=%dq" % (n + 1), *[0] * (n + 1))
        assert kvc.STATUS[call(which, words, n + 1, None)] == "KVC_ERR_INVALID"
        assert f"{n} arguments" in kvc._lib.kvc_last_error_string().decode()
    assert kvc.STATUS[call(21, words, 1, None)] == "KVC_ERR_INVALID"


def test_host_tensors_and_wrong_shapes_are_refused():
    t = lambda dt, *shape: torch.zeros(shape, dtype=dt)  # noqa: E731
    f16, f32, i32, i64, f8 = torch.float16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn
    tables = lambda **c: kvc.kv_block_tables(*{**dict(before=None, after=t(i32, 2), free=t(i32, 4), placed=t(i32, 1),  # noqa: E731
                                                      table=t(i32, 2, 4), new=t(i32, 1), cu=t(i32, 3), slots=t(i64, 8)),
                                               **c}.values())
    append = lambda **c: kvc.kv_append_fp8_block(*{**dict(k=t(f16, 3, 2, 64), v=t(f16, 3, 2, 64), slots=t(i64, 3),  # noqa: E731
                                                          codes=t(f8, 4, 2, 2, 16, 64), scales=t(f32, 4, 2, 2)), **c}.values())
    fp8 = lambda **c: kvc.paged_decode_attention_fp8_block(*{**dict(  # noqa: E731
        q=t(f16, 1, 4, 64), codes=t(f8, 4, 2, 2, 16, 64), scales=t(f32, 4, 2, 2), table=t(i32, 1, 4), ctx=t(i32, 1), scale=1.0,
        out=t(f16, 1, 4, 64), ws=None, most=64), **c}.values())
    window = lambda **c: kvc.paged_decode_window_attention(*{**dict(  # noqa: E731
        q=t(f16, 1, 4, 64), k=t(f16, 4, 2, 16, 64), v=t(f16, 4, 2, 16, 64), table=t(i32, 1, 4), ctx=t(i32, 1), window=4,
        sinks=0, scale=1.0, out=t(f16, 1, 4, 64), ws=None, most=64, kn=None, vn=None), **c}.values())
    prefill = lambda **c: kvc.prefill_window_attention(*{**dict(  # noqa: E731
        q=t(f16, 5, 4, 64), k=t(f16, 5, 2, 64), v=t(f16, 5, 2, 64), cu=t(i32, 2), most=5, window=4, sinks=0, scale=1.0,
        out=t(f16, 5, 4, 64)), **c}.values())
    for call in (tables, append, fp8, window, prefill):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    for call, change, kind in (
            (tables, dict(after=t(i32, 3)), ValueError), (tables, dict(cu=t(i32, 2)), ValueError),
            (tables, dict(placed=t(i32, 2)), ValueError), (tables, dict(table=t(i32, 8)), ValueError),
            (append, dict(v=t(f16, 3, 2, 128)), ValueError), (append, dict(slots=t(i64, 4)), ValueError),
            (append, dict(codes=t(f16, 4, 2, 2, 16, 64)), TypeError), (append, dict(codes=t(f8, 4, 3, 2, 16, 64)), ValueError),
            (append, dict(scales=t(f32, 4, 2)), ValueError), (fp8, dict(codes=t(f8, 4, 2, 16, 64)), ValueError),
            (fp8, dict(out=t(i32, 1, 4, 64)), TypeError), (fp8, dict(ctx=t(i32, 2)), ValueError),
            (window, dict(kn=t(f16, 1, 2, 64)), ValueError), (window, dict(kn=t(f16, 1, 4, 64), vn=t(f16, 1, 4, 64)), ValueError),
            (window, dict(out=t(f16, 1, 4, 128)), ValueError), (prefill, dict(v=t(f16, 5, 4, 64)), ValueError),
            (prefill, dict(out=t(torch.float64, 5, 4, 64)), TypeError)):
        with pytest.raises(kind):
            call(**change)
