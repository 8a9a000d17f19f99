"""The measured cases of one step of tree-drafted decoding over the paged cache.

A step drafts a tree of tokens for every sequence (node 0 is the newest sampled token, every other node's parent has a
smaller index), and runs, per layer, ``kv_append_rope`` (query / key norm, position rotation, rows into the cache) and
``paged_decode_tree_attention``; then once ``draft_tree_verify`` (which drafted tokens the target keeps, and the next
token) and ``kv_tree_commit`` (the kept nodes' cache rows move to the end of the sequence's context).

Where ``own`` is false, ``run`` computes the same in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

BS = 16  # tokens per cache block
HEADS = [(14, 2, 64), (32, 8, 128), (8, 8, 64), (16, 2, 128), (12, 4, 64)]  # query heads, KV heads, head dim


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one sequence's next token, 14 / 2 heads: one decode step of a chat, where the launch is the cost
        {"name": "append_one_token", "op": "append", "n": 1, "hq": 14, "hkv": 2, "d": 64, "rot": 64, "inter": False,
         "norm": True},
        # a serving step: 32 sequences x 16 tree nodes
        {"name": "append_serving_step", "op": "append", "n": 512, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "inter": False, "norm": True},
        # an odd number of prompt tokens, rotation of half the dims in adjacent pairs, no norm
        {"name": "append_odd_prompt", "op": "append", "n": 1923, "hq": 14, "hkv": 2, "d": 64, "rot": 32,
         "inter": True, "norm": False},
        # four prompts of 4096 tokens
        {"name": "append_prompts", "op": "append", "n": 16384, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "inter": False, "norm": True},
        # a chat's drafted tree of 8 nodes
        {"name": "tree_one_sequence", "op": "tree", "b": 1, "t": 8, "hq": 14, "hkv": 2, "d": 64, "ctx": 2048,
         "branch": 2, "ragged": False},
        # the serving step: 32 sequences of about 2048 tokens, trees of up to 16 nodes
        {"name": "tree_serving_step", "op": "tree", "b": 32, "t": 16, "hq": 14, "hkv": 2, "d": 64, "ctx": 2048,
         "branch": 2, "ragged": True},
        # wide trees (64 nodes x 4 query heads per KV head = 256 query rows)
        {"name": "tree_wide", "op": "tree", "b": 8, "t": 64, "hq": 32, "hkv": 8, "d": 128, "ctx": 4096,
         "branch": 4, "ragged": False},
        # long documents
        {"name": "tree_long_context", "op": "tree", "b": 4, "t": 16, "hq": 32, "hkv": 8, "d": 128, "ctx": 65536,
         "branch": 3, "ragged": True},
        # a chat's drafted chain over a small vocabulary
        {"name": "verify_one_sequence", "op": "verify", "b": 1, "t": 8, "v": 32000, "branch": 1, "distinct": False,
         "half": False},
        # a serving step, distinct children per node, a vocabulary that is a multiple of nothing
        {"name": "verify_serving_step", "op": "verify", "b": 64, "t": 16, "v": 128257, "branch": 3, "distinct": True,
         "half": False},
        # one sequence's accepted path, 24 layers
        {"name": "commit_one_sequence", "op": "commit", "l": 24, "b": 1, "t": 8, "hkv": 2, "d": 64, "ctx": 400},
        # the serving step's accepted paths, trees of 64 nodes
        {"name": "commit_serving_step", "op": "commit", "l": 24, "b": 64, "t": 64, "hkv": 8, "d": 128, "ctx": 300},
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "verify", "commit"])
    hq, hkv, d = rng.choice(HEADS)
    if op == "append":
        return {"op": op, "n": _spread(rng, 1, 16384), "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d // 2, 16]), "inter": rng.random() < 0.3, "norm": rng.random() < 0.7}
    if op == "tree":
        b, t = _spread(rng, 1, 64), _spread(rng, 1, 64)
        tokens = 4 * 65536 * 8 * 128 // (b * hkv * d)  # no more cache bytes, nor scores, than the largest listed
        scores = 4 * 32 * 16 * 65536 // (b * t * hq)
        return {"op": op, "b": b, "t": t, "hq": hq, "hkv": hkv, "d": d,
                "ctx": _spread(rng, t, max(t, min(65536, tokens, scores))), "branch": rng.randint(1, 5),
                "ragged": rng.random() < 0.5}
    if op == "verify":
        return {"op": op, "b": _spread(rng, 1, 64), "t": rng.randint(1, 16), "v": _spread(rng, 500, 128257),
                "branch": rng.randint(1, 5), "distinct": rng.random() < 0.5, "half": rng.random() < 0.3}
    return {"op": op, "l": rng.randint(1, 24), "b": _spread(rng, 1, 64), "t": rng.randint(4, 64), "hkv": hkv, "d": d,
            "ctx": rng.randint(64, 300)}


# ---------------------------------------------------------------- inputs
def _lens(case):
    """Tree sizes and context lengths (tree included) of every sequence."""
    b, t, ctx = case["b"], case["t"], case["ctx"]
    i = np.arange(b)
    if not case.get("ragged"):
        return np.full(b, t), np.full(b, ctx)
    tree = t - (i * 5) % (t // 2 + 1)
    return tree, np.maximum(tree, ctx - (i * 37) % (ctx // 4 + 1))


def _parents(t, branch, rng):
    """Parents of a tree of t nodes in breadth-first order: about `branch` children for a node (1: a chain)."""
    par = np.full(t, -1, np.int32)
    for j in range(1, t):
        par[j] = max(0, (j - 1) // branch - (int(rng.integers(0, 2)) if branch > 1 else 0))
    return par


def _masks(parents):
    """Per node, the bits of itself and its ancestors."""
    bits = [0] * len(parents)
    for j, p in enumerate(parents):
        bits[j] = (1 << j) | (bits[p] if p >= 0 else 0)
    return np.array([x - (1 << 64) if x >> 63 else x for x in bits], np.int64)


def _table(b, nblk, rng):
    """Physical blocks of b sequences, nblk each, in a permuted order; and the number of blocks."""
    n = b * nblk
    return rng.permutation(n).astype(np.int32).reshape(b, nblk), n


def _path_lens(case):
    """Nodes on every sequence's accepted path, the root among them: 1 to 8, as many as fit beside their sources."""
    most = min(8, (case["t"] + 1) // 2)
    return 1 + np.arange(case["b"]) * 3 % most if case["b"] > 1 else np.array([min(4, most)])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    on = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    normal = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731
    half = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.float16)  # noqa: E731
    st = {"case": case}
    op = case["op"]
    if op == "append":
        n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
        st["qkv"] = half(n, (hq + 2 * hkv) * d)  # the projections' output: a token's query, key and value rows
        st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, d)) for x in st["qkv"].split((hq * d, hkv * d, hkv * d), 1))
        st["qw"] = (1 + 0.2 * normal(d)).half() if case["norm"] else None
        st["kw"] = (1 + 0.2 * normal(d)).half() if case["norm"] else None
        st["eps"] = 1e-6
        st["freq"] = 1e4 ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
        st["pos"] = on((int(rng.integers(0, 100000)) + np.arange(n)).astype(np.int32))
        nb = -(-n // BS) + 8
        st["slots"] = on(rng.permutation(nb)[:-(-n // BS)].astype(np.int64).repeat(BS)[:n] * BS + np.arange(n) % BS)
        st["k_cache"], st["v_cache"] = half(nb, hkv, BS, d), half(nb, hkv, BS, d)
        st["q_out"] = torch.zeros(n, hq, d, dtype=torch.float16, device=dev)
    elif op == "tree":
        b, t, hq, hkv, d = (case[x] for x in ("b", "t", "hq", "hkv", "d"))
        tree, ctx = _lens(case)
        table, nb = _table(b, -(-case["ctx"] // BS), rng)
        st["k_cache"], st["v_cache"] = half(nb, hkv, BS, d), half(nb, hkv, BS, d)
        st["q"] = half(b, t, hq, d)
        st["table"], st["ctx"], st["tree"] = on(table), on(ctx.astype(np.int32)), on(tree.astype(np.int32))
        st["masks"] = on(np.stack([_masks(_parents(t, case["branch"], rng)) for _ in range(b)]))
        st["scale"] = d ** -0.5
        st["out"] = torch.zeros(b, t, hq, d, dtype=torch.float16, device=dev)
    elif op == "verify":
        b, t, v = case["b"], case["t"], case["v"]
        par = np.stack([_parents(t, case["branch"], rng) for _ in range(b)])
        rank = np.array([[int(np.sum(p[1:j] == p[j])) if j else 0 for j in range(t)] for p in par])
        dtype = torch.float16 if case["half"] else torch.float32
        st["p"], st["q"] = (torch.empty(b, t, v, dtype=dtype, device=dev) for _ in range(2))
        tok = torch.zeros(b, t, dtype=torch.int64, device=dev)
        for i in range(b):
            logits = 2.5 * normal(t, v)
            st["p"][i] = torch.softmax(logits, -1)
            draft = logits + 0.7 * normal(t, v)
            st["q"][i] = torch.softmax(draft, -1)
            par_i = on(par[i].clip(0)).long()
            # tokens drawn from their parent's row: the largest of log q + Gumbel noise, and for distinct children
            # the largest, the second largest, ... of the same noise
            gumbel = -torch.log(-torch.log(torch.rand(t, v, generator=gen, device=dev).clamp(1e-20, 1 - 1e-7)))
            if case["distinct"]:
                best = (draft + gumbel).topk(min(v, int(rank[i].max()) + 1), -1).indices
                tok[i] = best[par_i, on(rank[i])]
            else:
                tok[i] = (draft[par_i] + gumbel).argmax(-1)
        st["tokens"], st["parents"] = tok.int(), on(par)
        st["u"] = torch.rand(b, t, generator=gen, device=dev)
        st["path"] = torch.zeros(b, t, dtype=torch.int32, device=dev)
        st["path_len"], st["next"] = (torch.zeros(b, dtype=torch.int32, device=dev) for _ in range(2))
    else:
        lay, b, t, hkv, d = (case[x] for x in ("l", "b", "t", "hkv", "d"))
        nblk = -(-(case["ctx"] + t) // BS)
        table, nb = _table(b, nblk, rng)
        st["k_pool"], st["v_pool"] = half(lay, nb, hkv, BS, d), half(lay, nb, hkv, BS, d)
        plen = _path_lens(case)
        path = np.full((b, t), -1, np.int32)
        path[:, 0] = 0
        for i in range(b):  # sources behind every destination, so that a second pass moves the same rows again
            path[i, 1:plen[i]] = np.sort(rng.choice(np.arange(plen[i], t), plen[i] - 1, replace=False))
        st["table"], st["path"], st["path_len"] = on(table), on(path), on(plen.astype(np.int32))
        st["ctx"] = on((t + rng.integers(0, case["ctx"], b)).astype(np.int32))
        st["deep"] = int(plen.max())
        st["new_ctx"] = torch.zeros(b, dtype=torch.int32, device=dev)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"append": _own_append, "tree": _own_tree, "verify": _own_verify, "commit": _own_commit}[op](st)
    return {"append": _plain_append, "tree": _plain_tree, "verify": _plain_verify, "commit": _plain_commit}[op](st)


def _once(st, key, make):
    if key not in st:
        st[key] = make()
    return st[key]


def _own_append(st):
    import paged_kv_cache_27_gb300 as kvc
    turns = _once(st, "turns", lambda: torch.from_numpy(kvc.kv_rope_turns(st["freq"])).cuda())
    kvc.kv_append_rope(st["q"], st["k"], st["v"], st["pos"], turns, st["q_out"], st["k_cache"], st["v_cache"],
                       st["slots"], q_weight=st["qw"], k_weight=st["kw"], eps=st["eps"],
                       interleaved=st["case"]["inter"])
    return st["q_out"], st["k_cache"], st["v_cache"]


def _own_tree(st):
    import paged_kv_cache_27_gb300 as kvc
    b, t, hq, d = st["q"].shape
    hkv, most = st["case"]["hkv"], st["case"]["ctx"]
    ws = _once(st, "ws", lambda: torch.empty(max(16, kvc.paged_decode_tree_plan(b, hq, hkv, d, most, t)),
                                             dtype=torch.uint8, device="cuda"))
    kvc.paged_decode_tree_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["ctx"], st["masks"],
                                    st["scale"], st["out"], ws, most, tree_lens=st["tree"])
    return st["out"]


def _own_verify(st):
    import paged_kv_cache_27_gb300 as kvc
    kvc.draft_tree_verify(st["p"], st["q"], st["tokens"], st["parents"], st["u"], st["path"], st["path_len"],
                          st["next"], distinct=st["case"]["distinct"])
    return st["path"], st["path_len"], st["next"]


def _own_commit(st):
    import paged_kv_cache_27_gb300 as kvc
    lay, nb, hkv, _, d = st["k_pool"].shape
    h = _once(st, "h", lambda: kvc.kv_cache_create(kvc.KvcConfig(lay, nb, hkv, d), st["k_pool"], st["v_pool"]))
    kvc.kv_tree_commit(h, st["table"], st["ctx"], st["path"], st["path_len"], st["new_ctx"])
    return st["k_pool"], st["v_pool"], st["new_ctx"]


def _plain_append(st):
    case, rot = st["case"], st["case"]["rot"]
    # angles of far positions need 64 bits
    angle = st["pos"].double()[:, None] * torch.from_numpy(st["freq"]).cuda()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rows(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * w.float()
        r, rest = x[..., :rot], x[..., rot:]
        a, b = (r[..., 0::2], r[..., 1::2]) if case["inter"] else (r[..., :rot // 2], r[..., rot // 2:])
        c, s = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((c, s), -1).flatten(-2) if case["inter"] else torch.cat((c, s), -1)
        return torch.cat((r, rest), -1).half()

    blk, off = st["slots"] // BS, st["slots"] % BS
    st["k_cache"][blk, :, off] = rows(st["k"], st["kw"])
    st["v_cache"][blk, :, off] = st["v"]
    return rows(st["q"], st["qw"]), st["k_cache"], st["v_cache"]


def _plain_tree(st):
    b, t, hq, d = st["q"].shape
    hkv = st["case"]["hkv"]
    gather = lambda c: c[st["table"]].transpose(1, 2).flatten(2, 3).float()  # noqa: E731  [b][hkv][positions][d]
    k, v = gather(st["k_cache"]), gather(st["v_cache"])
    q = st["q"].float().view(b, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)  # [b][hkv][g][t][d]
    s = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).view(b, hkv, hq // hkv, t, -1) * st["scale"]
    pos = torch.arange(k.shape[2], device=k.device)
    node = pos[None] - (st["ctx"] - st["tree"])[:, None]  # [b][positions]: negative in the history
    in_tree = (node >= 0) & (node < st["tree"][:, None])
    seen = (st["masks"][:, :, None] >> node.clamp(0, 63)[:, None]) & 1 == 1
    valid = ((node < 0)[:, None] | (in_tree[:, None] & seen))[:, None, None]
    m = s.masked_fill(~valid, -math.inf).amax(-1, keepdim=True)
    e = torch.where(valid, torch.exp(s - torch.where(m.isfinite(), m, torch.zeros_like(m))), torch.zeros_like(s))
    o = torch.matmul(e.flatten(2, 3), v).view(b, hkv, hq // hkv, t, d)
    total = e.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(b, t, hq, d)
    live = torch.arange(t, device=k.device)[None] < st["tree"][:, None]  # rows behind a tree stay as they were
    return torch.where(live[:, :, None, None], o.half(), st["out"])


def _plain_verify(st):
    b, t, v = st["p"].shape
    p, q, u, par, tok = st["p"], st["q"], st["u"].double(), st["parents"].long(), st["tokens"].long()
    row = torch.arange(b, device=p.device)
    cur = torch.zeros(b, dtype=torch.int64, device=p.device)
    zero, one = torch.zeros(b, dtype=torch.float64, device=p.device), torch.ones(b, dtype=torch.float64, device=p.device)
    a, s, r = zero, one, one
    path = torch.full((b, t), -1, dtype=torch.int32, device=p.device)
    path[:, 0] = 0
    n = torch.ones_like(cur)
    # which node is tested next follows from the tests before it: one node after the other, all sequences at once
    for j in range(1, t):
        child = par[:, j] == cur
        pc, qc = p[row, cur, tok[:, j]].double(), q[row, cur, tok[:, j]].double()
        yes = child & (r > 0) & (u[:, j] * qc * s < (pc - a * qc).clamp_min(0) * r)
        no = child & ~yes
        a = torch.where(yes, zero, torch.where(no & (r > 0), a + s / r, a))
        if st["case"]["distinct"]:
            r = torch.where(yes, one, torch.where(no, r - qc, r))
        cur = torch.where(yes, torch.full_like(cur, j), cur)
        path.scatter_(1, torch.where(yes, n, n - 1)[:, None],
                      torch.where(yes, torch.full_like(cur, j), path.gather(1, (n - 1)[:, None])[:, 0].long())
                      .int()[:, None])
        n = n + yes
        left = (p[row, cur].double() - a[:, None] * q[row, cur].double()).clamp_min(0).sum(-1)
        s = torch.where(yes, one, torch.where(no, left, s))
    p_cur = p[row, cur].double()
    w = (p_cur - a[:, None] * q[row, cur].double()).clamp_min(0)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p_cur)
    c = w.cumsum(-1)
    nxt = (c <= (u[:, 0] * c[:, -1])[:, None]).sum(-1)
    return path, n.int(), nxt.int()


def _plain_commit(st):
    t, deep = st["path"].shape[1], st["deep"]  # no path is longer than the tree is deep
    base = (st["ctx"] - t)[:, None]
    j = torch.arange(deep, device=base.device)[None]
    moved = j < st["path_len"][:, None]
    to, frm = base + j, base + torch.where(moved, st["path"][:, :deep], j.int())  # rows behind a path: onto themselves
    tb = st["table"]
    blk_to, blk_from = tb.gather(1, (to // BS).long()), tb.gather(1, (frm // BS).long())
    for pool in (st["k_pool"], st["v_pool"]):
        pool[:, blk_to, :, to % BS] = pool[:, blk_from, :, frm % BS]
    return st["k_pool"], st["v_pool"], (st["ctx"] - t + st["path_len"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "append":
        n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
        return {"bytes": 2 * n * (hq + 2 * hkv) * d * 2 + n * 12 + 4 * d, "flops": n * (hq + hkv) * d * 7}
    if op == "tree":
        tree, ctx = _lens(case)
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        rows = int(tree.sum()) * hq
        return {"bytes": int(ctx.sum()) * hkv * d * 4 + rows * d * 4 + int((-(-ctx // BS)).sum()) * 4 + rows // hq * 8,
                "flops": int((tree * ctx).sum()) * hq * d * 4}
    if op == "verify":  # the target's and the draft's row of one node of every sequence
        n = case["b"] * case["v"]
        return {"bytes": n * (4 if case["half"] else 8) + case["b"] * case["t"] * 24, "flops": 4 * n}
    moved = int((_path_lens(case) - 1).sum())
    return {"bytes": moved * case["l"] * case["hkv"] * case["d"] * 2 * 2 * 2 + case["b"] * 16, "flops": 0}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    return {"append": _exact_append, "tree": _exact_tree, "verify": _exact_verify, "commit": _exact_commit}[op](st)


def _exact_append(st):
    case, d, rot = st["case"], st["case"]["d"], st["case"]["rot"]
    # rotation of the pair (x, y) by the angle g as the product (x + iy) e^(ig)
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                       torch.outer(st["pos"].double(), torch.from_numpy(st["freq"]).cuda()))[:, None]
    first = torch.arange(0, rot, 2, device="cuda") if case["inter"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if case["inter"] else rot // 2)

    def rows(x, w):
        y = x.double()
        if w is not None:
            y = y / (torch.linalg.vector_norm(y, dim=-1, keepdim=True).pow(2) / d + st["eps"]).sqrt() * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    k_rows, v_rows = (c.transpose(1, 2).flatten(0, 1).clone() for c in (k_cache, v_cache))
    k_rows[st["slots"]], v_rows[st["slots"]] = rows(st["k"], st["kw"]), st["v"].double()
    back = lambda x: x.unflatten(0, (-1, BS)).transpose(1, 2).contiguous()  # noqa: E731
    return rows(st["q"], st["qw"]), back(k_rows), back(v_rows)


def _exact_tree(st):
    b, t, hq, d = st["q"].shape
    hkv = st["case"]["hkv"]
    out = st["out"].double()
    masks = st["masks"].cpu().numpy().view(np.uint64)
    for i in range(b):
        ctx, tree = int(st["ctx"][i]), int(st["tree"][i])
        blocks = st["table"][i, :-(-ctx // BS)].long()
        allowed = np.ones((tree, ctx), bool)
        for node in range(tree):
            allowed[node, ctx - tree:] = [(int(masks[i, node]) >> other) & 1 for other in range(tree)]
        off = torch.from_numpy(~allowed).cuda()
        for h in range(hkv):
            k, v = (st[c][blocks, h].flatten(0, 1)[:ctx].double() for c in ("k_cache", "v_cache"))
            for g in range(h * hq // hkv, (h + 1) * hq // hkv):
                x = (st["q"][i, :tree, g].double() @ k.T * st["scale"]).masked_fill(off, -math.inf)
                out[i, :tree, g] = torch.softmax(x, -1).nan_to_num(0.0) @ v
    return out


def _exact_verify(st):
    b, t, v = st["p"].shape
    u, par, tok = (st[x].cpu().numpy() for x in ("u", "parents", "tokens"))
    path, length, nxt = np.full((b, t), -1, np.int32), np.zeros(b, np.int32), np.zeros(b, np.int32)
    for i in range(b):
        walk, node, going = [0], 0, True
        while going:
            going = False
            p, q = (st[x][i, node].cpu().numpy().astype(np.float64) for x in ("p", "q"))
            left, weight = p.copy(), 1.0  # the target's residual, and the draft's mass without the refused tokens
            whole = 1.0
            for c in np.flatnonzero(par[i] == node):
                if weight > 0 and float(u[i, c]) * q[tok[i, c]] / weight < left[tok[i, c]] / whole:
                    walk.append(int(c))
                    node, going = int(c), True
                    break
                if weight > 0:
                    left = np.maximum(left - whole * q / weight, 0.0)
                    whole = left.sum()
                if st["case"]["distinct"]:
                    weight -= q[tok[i, c]]
                if whole == 0:
                    left, whole = np.zeros_like(p), 0.0
                    break
            if not going:
                chosen = left if left.sum() > 0 else p
                sums = np.cumsum(chosen)
                nxt[i] = np.searchsorted(sums, float(u[i, 0]) * sums[-1], side="right")
        path[i, :len(walk)], length[i] = walk, len(walk)
    on = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return on(path), on(length), on(nxt)


def _exact_commit(st):
    t = st["path"].shape[1]
    table, path, ctx, n = (st[x].cpu().numpy() for x in ("table", "path", "ctx", "path_len"))
    k, v = st["k_pool"].double(), st["v_pool"].double()
    for i in range(len(n)):
        for j in range(int(n[i])):
            to, frm = int(ctx[i]) - t + j, int(ctx[i]) - t + int(path[i, j])
            for pool in (k, v):
                pool[:, table[i, to // BS], :, to % BS] = pool[:, table[i, frm // BS], :, frm % BS]
    return k, v, torch.from_numpy(ctx - t + n).cuda()
