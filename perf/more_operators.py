"""The measured cases of serving with windows and with an 8-bit cache, both over the paged cache.

A step of a serving loop has its request lengths on the GPU.  ``kv_block_tables`` gives every sequence the blocks that
its new tokens need and the slots where they go; ``kv_append_fp8_block`` writes their keys and values to an e4m3 cache
with one power-of-two scale per (block of tokens, KV head), and ``paged_decode_attention_fp8_block`` attends over it.
Where a model sees a sliding window and a few first tokens only, ``prefill_window_attention`` runs its prompts and
``paged_decode_window_attention`` its single tokens; the blocks of such a sequence are used in turn, so that its cache
holds no more than the window.

Where ``own`` is false, ``run`` computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

BS = 16  # tokens per cache block
HEADS = [(14, 2, 64), (32, 8, 128), (8, 8, 64), (16, 2, 128), (12, 4, 64)]  # query heads, KV heads, head dim
LEAST = -32  # exponent of the scale of a block of zeros
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's bookkeeping: 256 running sequences get one token each
        {"name": "tables_decode_step", "op": "tables", "b": 256, "fresh": False, "len": 2048, "new": 1, "window": 0,
         "sinks": 0},
        # prompts of up to 8192 tokens admitted at once, for a model with a window of 1024 and 4 sinks
        {"name": "tables_prompts", "op": "tables", "b": 128, "fresh": True, "len": 8192, "new": 8192, "window": 1024,
         "sinks": 4},
        # the rows of a decode step: 32 tokens, each somewhere inside its sequence's newest block
        {"name": "append_decode_step", "op": "append", "n": 32, "runs": 1, "hkv": 2, "d": 64},
        # four prompts of 4096 tokens
        {"name": "append_prompts", "op": "append", "n": 16384, "runs": 4096, "hkv": 8, "d": 128},
        # one chat of 2048 tokens over the 8-bit cache: launch and latency
        {"name": "decode8_one_sequence", "op": "decode8", "b": 1, "hq": 14, "hkv": 2, "d": 64, "ctx": 2048,
         "ragged": False, "window": 0, "sinks": 0},
        # a decode step of 32 sequences of about 2048 tokens
        {"name": "decode8_serving_step", "op": "decode8", "b": 32, "hq": 14, "hkv": 2, "d": 64, "ctx": 2048,
         "ragged": True, "window": 0, "sinks": 0},
        # long documents
        {"name": "decode8_long_context", "op": "decode8", "b": 4, "hq": 32, "hkv": 8, "d": 128, "ctx": 65536,
         "ragged": True, "window": 0, "sinks": 0},
        # one long chat, of which the last 1024 tokens and the first 4 are seen
        {"name": "window_one_sequence", "op": "window", "b": 1, "hq": 14, "hkv": 2, "d": 64, "ctx": 20001,
         "ragged": False, "window": 1024, "sinks": 4, "append": False},
        # a decode step of 64 sequences with a window of 4096, its append fused
        {"name": "window_serving_step", "op": "window", "b": 64, "hq": 32, "hkv": 8, "d": 128, "ctx": 32768,
         "ragged": True, "window": 4096, "sinks": 4, "append": True},
        # a few uneven prompts
        {"name": "prefill_uneven_prompts", "op": "prefill", "lens": "592,1920,128,3200,1", "hq": 8, "hkv": 8, "d": 64,
         "window": 512, "sinks": 4},
        # four prompts of 4096 tokens
        {"name": "prefill_prompts", "op": "prefill", "lens": "4096,4096,4096,4096", "hq": 32, "hkv": 8, "d": 128,
         "window": 1024, "sinks": 4},
        # one document
        {"name": "prefill_document", "op": "prefill", "lens": "32768", "hq": 14, "hkv": 2, "d": 64, "window": 4096,
         "sinks": 20},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode8", "decode8", "window", "window", "prefill", "prefill"])
    hq, hkv, d = rng.choice(HEADS)
    if op == "tables":
        fresh = rng.random() < 0.5
        b = _spread(rng, 1, 1024)
        most = max(1, min(8192, 128 * 8192 // b))
        windowed = rng.random() < 0.5
        return {"op": op, "b": b, "fresh": fresh, "len": _spread(rng, 1, most),
                "new": _spread(rng, 1, most) if fresh else 1, "window": _spread(rng, 1, 4096) if windowed else 0,
                "sinks": rng.choice([0, 1, 4, 33]) if windowed else 0}
    if op == "append":
        n = _spread(rng, 1, 16384)
        step = n <= 512 and rng.random() < 0.5
        return {"op": op, "n": n, "runs": 1 if step else _spread(rng, max(1, n // 512), 4096), "hkv": hkv, "d": d}
    if op in ("decode8", "window"):
        b = _spread(rng, 1, 64)
        windowed = op == "window" or rng.random() < 0.3
        window, sinks = (_spread(rng, 1, 4096), rng.choice([0, 1, 4, 33])) if windowed else (0, 0)
        tokens = 4 * 65536 * 8 * 128 // (b * hkv * d)  # no more cache bytes than the largest listed
        case = {"op": op, "b": b, "hq": hq, "hkv": hkv, "d": d,
                "ctx": _spread(rng, 1, 131072 if windowed else min(131072, tokens)), "ragged": rng.random() < 0.5,
                "window": window, "sinks": sinks}
        return {**case, "append": rng.random() < 0.4} if op == "window" else case
    window, left = _spread(rng, 1, 4096), 16384 * 1024 * 32 * 128
    lens = []
    for _ in range(rng.randint(1, 6)):
        lens.append(_spread(rng, 1, 8192))
        left -= lens[-1] * min(window, lens[-1]) * hq * d
        if left < 0:
            lens[-1] = 1 + lens[-1] % 128
            break
    return {"op": op, "lens": ",".join(map(str, lens)), "hq": hq, "hkv": hkv, "d": d, "window": window,
            "sinks": rng.choice([0, 1, 4, 33])}


# ---------------------------------------------------------------- inputs
def _context_lens(case):
    i = np.arange(case["b"])
    return np.maximum(1, case["ctx"] - (i * 37) % (case["ctx"] // 4 + 1)) if case["ragged"] else np.full_like(i, case["ctx"])


def _blocks(lens):
    return -(-lens // BS)


def _sink_blocks(case):
    return _blocks(case["sinks"]) if case["window"] else 0


def _ring(case):
    """Blocks that a window goes through in turn: it is never in more, wherever its last token lies in a block."""
    return _blocks(case["window"] + BS - 1) if case["window"] else 1 << 24


def _owned(case, blocks):
    """Distinct blocks behind the first `blocks` of a sequence."""
    return np.minimum(blocks, _sink_blocks(case) + _ring(case))


def _place(case, j):
    """Which of a sequence's distinct blocks its block j is."""
    first = _sink_blocks(case)
    return np.where(j < first + _ring(case), j, first + (j - first) % _ring(case))


def _table(case, ctx, rng):
    """The block table of sequences of these lengths, distinct blocks in a permuted order; and the number of blocks."""
    need = _owned(case, _blocks(ctx))
    start = np.cumsum(need) - need
    n = int(need.sum())
    ids = rng.permutation(n).astype(np.int32)
    j = np.arange(int(_blocks(ctx).max()))[None]
    place = np.where(j < _blocks(ctx)[:, None], start[:, None] + _place(case, j), 0)
    return np.where(j < _blocks(ctx)[:, None], ids[place], 0).astype(np.int32), n


def _table_lens(case):
    """Lengths before and after the step: sizes, like the others, and not drawn anew for other inputs."""
    rng = np.random.default_rng([case["b"], case["len"]])
    if case["fresh"]:
        after = rng.integers(1, case["new"] + 1, case["b"])
        after[0] = case["new"]
        return np.zeros_like(after), after
    before = rng.integers(max(1, case["len"] // 2), case["len"] + 1, case["b"])
    return before, before + case["new"]


def _quantize(x):
    """Codes and exponents of rows [..., BS, D], one exponent for a block: the least with no value beyond 448 of it."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax((-2, -1)))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, LEAST))
    return torch.ldexp(x, -e[..., None, None]).to(F8), e


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    half = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float16)  # noqa: E731
    st = {"case": case}
    op = case["op"]
    if op == "tables":
        before, after = _table_lens(case)
        most = int(_blocks(after).max()) + 1
        first = int(_owned(case, _blocks(before)).sum())
        spare = int((_owned(case, _blocks(after)) - _owned(case, _blocks(before))).sum())
        ids = rng.permutation(first + spare + 40).astype(np.int32)
        table = np.full((case["b"], most), -1, np.int32)
        if not case["fresh"]:
            held, at = _table(case, before, rng)
            table[:, :held.shape[1]] = np.where(np.arange(held.shape[1])[None] < _blocks(before)[:, None], ids[held], -1)
        placed = 7  # of the spare blocks, placed by earlier steps
        st["free"] = on(np.concatenate([rng.integers(0, 1 << 20, placed).astype(np.int32), ids[first:]]))
        st["placed"] = on(np.array([placed], np.int32))
        st["before"] = None if case["fresh"] else on(before.astype(np.int32))
        st["after"], st["table"] = on(after.astype(np.int32)), on(table)
        n = int((after - before).sum()) + 13  # a step's buffers have a fixed size, and are rarely full
        st["new_placed"] = torch.zeros(1, dtype=torch.int32, device=dev)
        st["cu"] = torch.zeros(case["b"] + 1, dtype=torch.int32, device=dev)
        st["slots"] = torch.zeros(n, dtype=torch.int64, device=dev)
        st["positions"] = torch.zeros(n, dtype=torch.int32, device=dev)
    elif op == "append":
        n, hkv, d = case["n"], case["hkv"], case["d"]
        # runs of tokens at the end of sequences that hold 0 to 2 blocks before them
        counts = np.full(-(-n // case["runs"]), case["runs"])
        counts[-1] = n - counts[:-1].sum()
        old = rng.integers(0, 2 * BS + 1, len(counts))
        need = _blocks(old + counts)
        start = np.cumsum(need) - need
        nb = int(_blocks(2 * BS + counts).sum())
        ids = rng.permutation(nb)
        seq = np.repeat(np.arange(len(counts)), counts)
        pos = old[seq] + np.arange(n) - (np.cumsum(counts) - counts)[seq]
        st["slots"] = on((ids[start[seq] + pos // BS] * BS + pos % BS).astype(np.int64))
        size = torch.exp2(torch.rand(n, hkv, 1, generator=gen, device=dev) * 4 - 2).half()
        rows = torch.cat((half(n, hkv, d) * size, half(n, hkv, d)), 1)  # a projection's key and value rows
        st["k"], st["v"] = rows[:, :hkv], rows[:, hkv:]
        codes, e = _quantize(half(nb, hkv, 2, BS, d) * torch.exp2(torch.rand(nb, hkv, 2, 1, 1, generator=gen, device=dev) * 4 - 2).half())
        st["codes"], st["scales"] = codes, torch.exp2(e.float())
    elif op in ("decode8", "window"):
        b, hq, hkv, d = case["b"], case["hq"], case["hkv"], case["d"]
        ctx = _context_lens(case)
        table, nb = _table(case, ctx, rng)
        st["table"], st["ctx"] = on(table), on(ctx.astype(np.int32))
        st["q"], st["scale"] = half(b, hq, d), d ** -0.5
        st["out"] = torch.zeros(b, hq, d, dtype=torch.float16, device=dev)
        if op == "decode8":
            st["codes"] = torch.empty(nb, hkv, 2, BS, d, dtype=F8, device=dev)
            st["scales"] = torch.empty(nb, hkv, 2, device=dev)
            for i in range(0, nb, 4096):
                part = half(min(4096, nb - i), hkv, 2, BS, d)
                part *= torch.exp2(torch.rand(*part.shape[:3], 1, 1, generator=gen, device=dev) * 2 - 1).half()
                st["codes"][i:i + 4096], e = _quantize(part)
                st["scales"][i:i + 4096] = torch.exp2(e.float())
        else:
            st["k_cache"], st["v_cache"] = half(nb, hkv, BS, d), half(nb, hkv, BS, d)
            if case["append"]:
                st["k_new"], st["v_new"] = half(b, hkv, d), half(b, hkv, d)
    else:
        lens = [int(x) for x in case["lens"].split(",")]
        n, hq, hkv, d = sum(lens), case["hq"], case["hkv"], case["d"]
        st["lens"] = lens
        st["cu"] = on(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        st["q"], st["k"], st["v"] = half(n, hq, d), half(n, hkv, d), half(n, hkv, d)
        st["scale"] = d ** -0.5
        st["out"] = torch.zeros(n, hq, d, dtype=torch.float16, device=dev)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "decode8": _own_decode8, "window": _own_window,
                "prefill": _own_prefill}[op](st)
    return {"tables": _plain_tables, "append": _plain_append, "decode8": _plain_decode8, "window": _plain_window,
            "prefill": _plain_prefill}[op](st)


def _once(st, key, make):
    if key not in st:
        st[key] = make()
    return st[key]


def _own_tables(st):
    import paged_kv_cache_27_gb300 as kvc
    kvc.kv_block_tables(st["before"], st["after"], st["free"], st["placed"], st["table"], st["new_placed"], st["cu"],
                        st["slots"], st["positions"], window=st["case"]["window"], sinks=st["case"]["sinks"])
    return st["table"], st["new_placed"], st["cu"], st["slots"], st["positions"]


def _own_append(st):
    import paged_kv_cache_27_gb300 as kvc
    kvc.kv_append_fp8_block(st["k"], st["v"], st["slots"], st["codes"], st["scales"])
    return st["codes"], st["scales"]


def _own_decode8(st):
    import paged_kv_cache_27_gb300 as kvc
    case = st["case"]
    (b, hq, d), hkv, most, window, sinks = st["q"].shape, case["hkv"], case["ctx"], case["window"], case["sinks"]
    ws = _once(st, "ws", lambda: torch.empty(
        max(16, kvc.paged_decode_fp8_block_plan(b, hq, hkv, d, most, window=window, sinks=sinks)), dtype=torch.uint8,
        device="cuda"))
    kvc.paged_decode_attention_fp8_block(st["q"], st["codes"], st["scales"], st["table"], st["ctx"], st["scale"],
                                         st["out"], ws, most, window=window, sinks=sinks)
    return st["out"]


def _own_window(st):
    import paged_kv_cache_27_gb300 as kvc
    case = st["case"]
    (b, hq, d), hkv, most, window, sinks = st["q"].shape, case["hkv"], case["ctx"], case["window"], case["sinks"]
    ws = _once(st, "ws", lambda: torch.empty(max(16, kvc.paged_decode_window_plan(b, hq, hkv, d, most, window, sinks)),
                                             dtype=torch.uint8, device="cuda"))
    new = {"k_new": st["k_new"], "v_new": st["v_new"]} if case["append"] else {}
    kvc.paged_decode_window_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["ctx"], window, sinks,
                                      st["scale"], st["out"], ws, most, **new)
    return (st["out"], st["k_cache"], st["v_cache"]) if case["append"] else st["out"]


def _own_prefill(st):
    import paged_kv_cache_27_gb300 as kvc
    kvc.prefill_window_attention(st["q"], st["k"], st["v"], st["cu"], max(st["lens"]), st["case"]["window"],
                                 st["case"]["sinks"], st["scale"], st["out"])
    return st["out"]


def _plain_tables(st):
    case, after, table = st["case"], st["after"].long(), st["table"]
    before = torch.zeros_like(after) if st["before"] is None else st["before"].long()
    first, ring = _sink_blocks(case), _ring(case)
    nb0, nb1 = (before + BS - 1) // BS, (after + BS - 1) // BS
    had = nb0.clamp(max=first + ring)
    need = nb1.clamp(max=first + ring) - had
    start = st["placed"].long() + need.cumsum(0) - need
    j = torch.arange(table.shape[1], device=table.device)[None]
    place = torch.where(j < first + ring, j, first + (j - first) % ring).expand(table.shape)
    fresh = st["free"][(start[:, None] + place - had[:, None]).clamp(0, len(st["free"]) - 1)]
    entry = torch.where(place < had[:, None], table.gather(1, place), fresh)
    new = (j >= nb0[:, None]) & (j < nb1[:, None])
    table.copy_(torch.where(new, entry, table))
    count = after - before
    cu = torch.cat((torch.zeros_like(count[:1]), count.cumsum(0)))
    t = torch.arange(len(st["slots"]), device=table.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    live = seq < len(count)
    seq = seq.clamp(max=len(count) - 1)
    pos = torch.where(live, before[seq] + t - cu[seq], 0)
    kept = live & ((pos // BS < first) | (pos // BS + ring >= nb1[seq]))
    slots = torch.where(kept, table[seq, pos // BS].long() * BS + pos % BS, -1)
    return table, (st["placed"] + need.sum()).int(), cu.int(), slots, pos.int()


def _plain_append(st):
    codes, scales = st["codes"], st["scales"]
    blk, off = st["slots"] // BS, st["slots"] % BS
    rows = torch.stack((st["k"], st["v"]), 2).float()  # [n][hkv][2][d]
    nb, hkv = codes.shape[:2]
    top = torch.zeros(nb, hkv, 2, device=rows.device)
    top.index_reduce_(0, blk, rows.abs().amax(-1), "amax")
    start = torch.full((nb,), BS, dtype=torch.int64, device=rows.device).index_reduce_(0, blk, off, "amin")
    m, e = torch.frexp(top)
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, LEAST))
    old = torch.frexp(scales)[1] - 1
    e = torch.where((start > 0)[:, None, None], torch.maximum(e, old), e)
    touched = torch.unique(blk)
    as_bytes = codes.view(torch.uint8)
    grown = torch.ldexp(as_bytes[touched].view(F8).float(), (old - e)[touched][..., None, None]).to(F8)
    keep = (torch.arange(BS, device=blk.device)[None] < start[touched][:, None])[:, None, None, :, None]
    as_bytes[touched] = torch.where(keep, grown.view(torch.uint8), as_bytes[touched])
    as_bytes[blk, :, :, off] = torch.ldexp(rows, -e[blk][..., None]).to(F8).view(torch.uint8)
    scales[touched] = torch.exp2(e[touched].float())
    return codes, scales


def _attend(st, ctx, table, gather):
    """Attention of one token of every sequence over its visible positions; gather(blocks) gives [b][hkv][n][d]."""
    case = st["case"]
    b, hq, d = st["q"].shape
    hkv, window, sinks = case["hkv"], case["window"], case["sinks"]
    # the blocks that can be seen: the sinks' first, and from the window's first to the last
    first = (ctx - window).clamp(min=0) if window else torch.zeros_like(ctx)
    width = min(table.shape[1], _blocks(window + BS - 1) if window else table.shape[1])
    lo = first // BS
    sink = torch.arange(min(table.shape[1], _sink_blocks(case)), device=ctx.device)[None].expand(b, -1)
    near = lo[:, None] + torch.arange(width, device=ctx.device)[None]
    j = torch.cat((sink, near), 1)
    pos = (j[:, :, None] * BS + torch.arange(BS, device=ctx.device)).flatten(1)
    is_sink = (torch.arange(j.shape[1], device=ctx.device) < sink.shape[1]).repeat_interleave(BS)[None]
    seen = torch.where(is_sink, (pos < sinks) & (pos < first[:, None]), (pos >= first[:, None]) & (pos < ctx[:, None]))
    k, v = gather(table.gather(1, j.clamp(max=table.shape[1] - 1)).long())
    q = st["q"].float().view(b, hkv, hq // hkv, d)
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    e = torch.exp(s - s.amax(-1, keepdim=True))
    return (torch.matmul(e, v) / e.sum(-1, keepdim=True)).view(b, hq, d).half()


def _plain_decode8(st):
    def gather(blocks):  # [b][blocks] -> the blocks' values
        c = st["codes"].view(torch.uint8)[blocks].view(F8).float() * st["scales"][blocks][..., None, None]  # [b][blocks][hkv][2][bs][d]
        return (c[:, :, :, i].transpose(1, 2).flatten(2, 3) for i in range(2))
    return _attend(st, st["ctx"].long(), st["table"], gather)


def _plain_window(st):
    ctx = st["ctx"].long()
    if st["case"]["append"]:
        last = ctx - 1
        blk = st["table"].gather(1, (last // BS)[:, None])[:, 0].long()
        st["k_cache"][blk, :, last % BS], st["v_cache"][blk, :, last % BS] = st["k_new"], st["v_new"]
    gather = lambda blocks: (c[blocks].transpose(1, 2).flatten(2, 3).float() for c in (st["k_cache"], st["v_cache"]))  # noqa: E731
    out = _attend(st, ctx, st["table"], gather)
    return (out, st["k_cache"], st["v_cache"]) if st["case"]["append"] else out


def _plain_prefill(st):
    case, n0 = st["case"], 0
    (n, hq, d), hkv, window, sinks = st["q"].shape, case["hkv"], case["window"], case["sinks"]
    out = torch.empty_like(st["out"])
    for length in st["lens"]:
        rows = slice(n0, n0 + length)
        q = st["q"][rows].float().view(length, hkv, hq // hkv, d).permute(1, 2, 0, 3)
        k, v = (st[x][rows].float().transpose(0, 1) for x in ("k", "v"))
        for r0 in range(0, length, 1024):  # the keys that 1024 rows can see: the sinks, and from the first row's window on
            r1 = min(length, r0 + 1024)
            lo = max(0, r0 - window + 1)
            first = min(sinks, lo)
            pos = torch.cat((torch.arange(first, device=k.device), torch.arange(lo, r1, device=k.device)))
            kk, vv = k[:, pos], v[:, pos]
            i = torch.arange(r0, r1, device=k.device)[:, None]
            seen = (pos <= i) & ((pos > i - window) | (pos < sinks))
            g = hq // hkv
            s = torch.matmul(q[:, :, r0:r1].flatten(1, 2), kk.transpose(-1, -2)).view(hkv, g, r1 - r0, -1) * st["scale"]
            s = s.masked_fill(~seen, -math.inf)
            e = torch.exp(s - s.amax(-1, keepdim=True))
            o = torch.matmul(e.flatten(1, 2), vv).view(hkv, g, r1 - r0, d) / e.sum(-1, keepdim=True)
            out[n0 + r0:n0 + r1] = o.permute(2, 0, 1, 3).reshape(r1 - r0, hq, d).half()
        n0 += length
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def _seen(case, ctx):
    """Positions that a sequence's newest token sees."""
    if not case["window"]:
        return ctx
    start = np.maximum(ctx - case["window"], 0)
    return ctx - start + np.minimum(case["sinks"], start)


def work(case):
    op = case["op"]
    if op == "tables":
        before, after = _table_lens(case)
        entries = int((_blocks(after) - _blocks(before)).sum())
        return {"bytes": 12 * (int((after - before).sum()) + 13) + 8 * entries + 12 * case["b"], "flops": 0}
    if op == "append":
        n, row = case["n"], case["hkv"] * case["d"]
        return {"bytes": n * row * 2 * 3 + n * 8, "flops": 4 * n * row}
    if op == "prefill":
        pairs = 0
        for length in (int(x) for x in case["lens"].split(",")):
            pairs += int(_seen(case, np.arange(1, length + 1)).sum())
        n, hq, hkv, d = sum(int(x) for x in case["lens"].split(",")), case["hq"], case["hkv"], case["d"]
        return {"bytes": n * (2 * hq + 2 * hkv) * d * 2, "flops": 4 * pairs * hq * d}
    seen = int(_seen(case, _context_lens(case)).sum())
    b, hq, hkv, d = case["b"], case["hq"], case["hkv"], case["d"]
    size = 1 if op == "decode8" else 2
    return {"bytes": seen * hkv * d * 2 * size + (seen // BS) * (8 * hkv * (2 - size) + 4) + b * hq * d * 4,
            "flops": 4 * seen * hq * d}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"tables": _exact_tables, "append": _exact_append, "decode8": _exact_decode, "window": _exact_decode,
            "prefill": _exact_prefill}[case["op"]](st)


def _exact_tables(st):
    case = st["case"]
    after, table, free = (st[x].cpu().numpy() for x in ("after", "table", "free"))
    before = np.zeros_like(after) if st["before"] is None else st["before"].cpu().numpy()
    at = int(st["placed"][0])
    slots, positions = np.full(len(st["slots"]), -1, np.int64), np.zeros(len(st["slots"]), np.int32)
    cu, t = [0], 0
    sink_blocks = -(-case["sinks"] // BS)
    turn = -(-(case["window"] + BS - 1) // BS)
    for i in range(case["b"]):
        held, blocks = -(-int(before[i]) // BS), -(-int(after[i]) // BS)
        for j in range(held, blocks):
            if case["window"] and j >= sink_blocks + turn:
                table[i, j] = table[i, j - turn]
            else:
                table[i, j] = free[at]
                at += 1
        for p in range(int(before[i]), int(after[i])):
            positions[t] = p
            j = p // BS
            if not case["window"] or j < sink_blocks or j >= blocks - turn:
                slots[t] = int(table[i, j]) * BS + p % BS
            t += 1
        cu.append(t)
    on = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return on(table), on(np.array([at], np.int32)), on(np.array(cu, np.int32)), on(slots), on(positions)


def _exact_append(st):
    codes, scales = st["codes"].double().cpu(), st["scales"].double().cpu()
    slots = st["slots"].cpu().numpy()
    rows = torch.stack((st["k"], st["v"]), 2).double().cpu()
    grid = torch.arange(256, dtype=torch.uint8).view(F8).double()
    grid = grid[grid.isfinite() & (grid >= 0)].sort().values.unique()  # what e4m3 holds; an even place is an even code

    def nearest(x):
        a = x.abs()
        up = torch.searchsorted(grid, a.contiguous()).clamp(max=len(grid) - 1)
        down = (up - 1).clamp(min=0)
        to_up, to_down = grid[up] - a, a - grid[down]
        place = torch.where((to_up < to_down) | ((to_up == to_down) & (up % 2 == 0)), up, down)
        return grid[place] * torch.sign(x)

    order = {}
    for t, s in enumerate(slots):
        order.setdefault(int(s) // BS, []).append((int(s) % BS, t))
    for blk, held in order.items():
        start = min(o for o, _ in held)
        new = rows[[t for _, t in held]]
        top = new.abs().amax((0, -1))
        e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), torch.tensor(float(LEAST), dtype=torch.float64))
        if start > 0:
            e = torch.maximum(e, torch.log2(scales[blk]))
            codes[blk, :, :, :start] = nearest(codes[blk, :, :, :start] * (scales[blk] / torch.exp2(e))[..., None, None])
        for o, t in held:
            codes[blk, :, :, o] = nearest(rows[t] / torch.exp2(e)[..., None])
        scales[blk] = torch.exp2(e)
    return codes.cuda(), scales.cuda()


def _exact_decode(st):
    case = st["case"]
    b, hq, d = st["q"].shape
    hkv, window, sinks = case["hkv"], case["window"], case["sinks"]
    ctx, table = st["ctx"].cpu().numpy(), st["table"].cpu().numpy()
    fp8 = case["op"] == "decode8"
    caches = () if fp8 else (st["k_cache"].clone(), st["v_cache"].clone())
    out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
    for i in range(b):
        n = int(ctx[i])
        if not fp8 and case["append"]:
            blk, off = int(table[i, (n - 1) // BS]), (n - 1) % BS
            caches[0][blk, :, off], caches[1][blk, :, off] = st["k_new"][i], st["v_new"][i]
        p = np.arange(n)
        if window:
            p = p[(p >= n - window) | (p < sinks)]
        blk, off = (torch.from_numpy(x.astype(np.int64)).cuda() for x in (table[i, p // BS], p % BS))
        for h in range(hkv):
            if fp8:
                k, v = (st["codes"].view(torch.uint8)[blk, h, c, off].view(F8).double() *
                        st["scales"][blk, h, c].double()[:, None] for c in (0, 1))
            else:
                k, v = (c[blk, h, off].double() for c in caches)
            g = slice(h * hq // hkv, (h + 1) * hq // hkv)
            out[i, g] = torch.softmax(st["q"][i, g].double() @ k.T * st["scale"], -1) @ v
    return (out, *(c.double() for c in caches)) if not fp8 and case["append"] else out


def _exact_prefill(st):
    case = st["case"]
    n, hq, d = st["q"].shape
    hkv, window, sinks = case["hkv"], case["window"], case["sinks"]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    at = 0
    for length in st["lens"]:
        for r in range(0, length, 512):
            i = torch.arange(r, min(length, r + 512), device="cuda")
            some = torch.arange(0, int(i[-1]) + 1, device="cuda")
            some = some[(some > r - window) | (some < sinks)]
            hidden = (some[None] > i[:, None]) | ((some[None] <= i[:, None] - window) & (some[None] >= sinks))
            for h in range(hq):
                kv = h * hkv // hq
                k, v = st["k"][at + some, kv].double(), st["v"][at + some, kv].double()
                x = (st["q"][at + i, h].double() @ k.T * st["scale"]).masked_fill(hidden, -math.inf)
                out[at + i, h] = torch.softmax(x, -1) @ v
        at += length
    return out
