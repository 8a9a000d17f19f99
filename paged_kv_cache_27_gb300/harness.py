"""Drives the library through its public API on the synthetic workloads.

Used by the benchmark and the GPU tests: it allocates pools and buffers with
PyTorch, fills caches through ``kv_append``, runs decode steps, the
serving-mix allocation protocol on the library's own block pool, and the
prefill-then-decode flow.  Every step calls the C ABI; nothing here computes
attention or slots itself.
"""
from __future__ import annotations

import numpy as np
import torch

from . import (KvcConfig, draft_tree_verify, kv_append, kv_append_fp8_block, kv_append_rope, kv_block_alloc,
               kv_block_release, kv_block_share, kv_block_tables, kv_cache_create, kv_cache_destroy, kv_copy_blocks,
               kv_rope_turns, kv_tree_commit, kv_tree_masks, kvc_copy_async, kv_slot_mapping, kv_step_prepare,
               paged_decode_append_attention, paged_decode_attention, paged_decode_attention_fp8_block,
               paged_decode_fp8_block_plan, paged_decode_plan, paged_decode_tree_attention, paged_decode_tree_plan,
               paged_decode_window_attention, paged_decode_window_plan, paged_decode_workspace_init, prefill_attention,
               prefill_window_attention)

F16_NAN = 0x7E00  # a quiet-NaN bit pattern used to poison cache slots nobody owns


def _dev(a, device, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    if dtype is not None:
        t = t.to(dtype)
    return t.to(device)


def poisoned_pool(shape, device) -> torch.Tensor:
    """fp16 pool filled with NaN bits: any read of a slot outside a context would show up."""
    return torch.full(shape, F16_NAN, dtype=torch.int16, device=device).view(torch.float16)


class DecodeSession:
    """A paged cache holding a DecodeWorkload's history, ready for decode steps on every layer."""

    def __init__(self, wl, device="cuda", out_dtype=torch.float32, blocks_per_split=0, poison=True):
        self.wl = wl
        self.device = device
        cfg = KvcConfig(num_layers=wl.L, num_blocks=wl.NB, num_kv_heads=wl.Hkv, head_dim=wl.D, block_size=wl.bs)
        self.cfg = cfg
        alloc = poisoned_pool if poison else (lambda s, d: torch.zeros(s, dtype=torch.float16, device=d))
        self.k_pool = alloc(cfg.pool_shape, device)
        self.v_pool = alloc(cfg.pool_shape, device)
        self.h = kv_cache_create(cfg, self.k_pool, self.v_pool)
        B = wl.B
        self.max_ctx = int(wl.ctx.max())
        self.block_table = _dev(wl.block_table, device)
        self.context_lens = _dev(wl.ctx, device)
        ones = np.ones(B, np.int32)
        self.hist_slots = _dev(kv_slot_mapping(wl.block_table, np.zeros(B, np.int32), wl.ctx - 1, wl.bs), device)
        self.step_slots_host = kv_slot_mapping(wl.block_table, wl.ctx - 1, ones, wl.bs)
        self.step_slots = _dev(self.step_slots_host, device)
        self.q = _dev(wl.q, device)
        self.k_new = _dev(wl.k_new, device)
        self.v_new = _dev(wl.v_new, device)
        self.out = torch.empty((wl.L, B, wl.Hq, wl.D), dtype=out_dtype, device=device)
        self.blocks_per_split = blocks_per_split
        self.nsplit, self.bps, ws = paged_decode_plan(B, wl.Hq, wl.Hkv, wl.D, self.max_ctx, blocks_per_split)
        self.workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=device)
        paged_decode_workspace_init(self.workspace)

    def fill(self):
        """Write every sequence's history (positions 0 .. ctx-2) into the cache, layer by layer."""
        for layer in range(self.wl.L):
            kh = _dev(self.wl.k_hist[layer], self.device)
            vh = _dev(self.wl.v_hist[layer], self.device)
            kv_append(self.h, layer, kh, vh, self.hist_slots)
        return self

    def append(self, layer, stream=None):
        kv_append(self.h, layer, self.k_new[layer], self.v_new[layer], self.step_slots, stream=stream)

    def decode(self, layer, stream=None):
        paged_decode_attention(self.q[layer], self.k_pool[layer], self.v_pool[layer], self.block_table,
                               self.context_lens, self.wl.scale, self.out[layer], self.workspace, self.max_ctx,
                               self.blocks_per_split, stream=stream)

    def decode_append(self, layer, stream=None):
        """Fused append + decode of one layer."""
        paged_decode_append_attention(self.q[layer], self.k_new[layer], self.v_new[layer], self.k_pool[layer],
                                      self.v_pool[layer], self.block_table, self.context_lens, self.wl.scale,
                                      self.out[layer], self.workspace, self.max_ctx, self.blocks_per_split,
                                      stream=stream)

    def step(self, stream=None, fused=False):
        """One decode step: for every layer, append the new token's K/V, then attend.

        fused=False: kv_append then paged_decode_attention; fused=True: paged_decode_append_attention."""
        for layer in range(self.wl.L):
            if fused:
                self.decode_append(layer, stream)
            else:
                self.append(layer, stream)
                self.decode(layer, stream)

    def capture(self, fused=True, decode_only=False, stream=None):
        """CUDA graph of one step (or of the 24 decode calls alone); eager warm-up first."""
        stream = stream or torch.cuda.Stream(self.device)
        with torch.cuda.stream(stream):
            self._graph_body(fused, decode_only)
        torch.cuda.synchronize(self.device)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            self._graph_body(fused, decode_only)
        torch.cuda.synchronize(self.device)
        return graph

    def _graph_body(self, fused, decode_only):
        if decode_only:
            for layer in range(self.wl.L):
                self.decode_append(layer) if fused else self.decode(layer)
        else:
            self.step(fused=fused)

    def close(self):
        if self.h:
            kv_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def serving_mix(mix, device="cuda", out_dtype=torch.float32, poison=True):
    """The serving-mix protocol on the library's block pool: groups of `mix.group` sequences share the blocks of a
    common prompt prefix (refcounted, allocated once per group), each sequence owns the blocks of its private
    tail, and one decode step appends a token per sequence — a sequence whose last block is shared gets a
    private copy first (copy-on-write) — and then runs paged decode over the new tables.

    Returns a dict: block tables before/after the step, copy pairs, slots, pools and the output."""
    bs = mix.bs
    cfg = KvcConfig(num_layers=1, num_blocks=mix.NB, num_kv_heads=mix.Hkv, head_dim=mix.D, block_size=bs)
    alloc = poisoned_pool if poison else (lambda s, d: torch.zeros(s, dtype=torch.float16, device=d))
    k_pool, v_pool = alloc(cfg.pool_shape, device), alloc(cfg.pool_shape, device)
    h = kv_cache_create(cfg, k_pool, v_pool)
    try:
        for _ in range(mix.NB):
            kv_block_alloc(h)
        for pid in mix.free_order:
            kv_block_release(h, int(pid))
        B, G = mix.B, mix.group
        npre = -(-mix.prefix_len // bs)
        tables = [[] for _ in range(B)]
        for g in range(-(-B // G)):
            members = range(g * G, min(B, (g + 1) * G))
            prefix_pages = [kv_block_alloc(h) for _ in range(npre)]
            for b in members:
                need = -(-min(mix.prefix_len, int(mix.ctx[b]) - 1) // bs)
                for pid in prefix_pages[:need]:
                    kv_block_share(h, pid)
                tables[b] = list(prefix_pages[:need])
            n_pre = max(min(mix.prefix_len, int(mix.ctx[b]) - 1) for b in members)
            slots = kv_slot_mapping(np.array([prefix_pages], np.int32), [0], [n_pre], bs)
            kv_append(h, 0, _dev(mix.prefix_k[g, :n_pre], device), _dev(mix.prefix_v[g, :n_pre], device),
                      _dev(slots, device))
            for pid in prefix_pages:
                kv_block_release(h, pid)
            for b in members:
                while len(tables[b]) * bs < int(mix.ctx[b]) - 1:
                    tables[b].append(kv_block_alloc(h))
                n_suf = int(mix.suffix_off[b + 1] - mix.suffix_off[b])
                if n_suf:
                    row = np.array([tables[b]], np.int32)
                    slots = kv_slot_mapping(row, [mix.prefix_len], [n_suf], bs)
                    sl = slice(int(mix.suffix_off[b]), int(mix.suffix_off[b + 1]))
                    kv_append(h, 0, _dev(mix.suffix_k[sl], device), _dev(mix.suffix_v[sl], device),
                              _dev(slots, device))
        tables_before = [list(t) for t in tables]
        mb = max(-(-int(c) // bs) for c in mix.ctx)
        table = np.full((B, mb), -1, np.int32)
        nblk = np.zeros(B, np.int32)
        for b in range(B):
            table[b, :len(tables[b])] = tables[b]
            nblk[b] = len(tables[b])
        slots, copies = kv_step_prepare(h, table, nblk, mix.ctx - 1)
        kv_copy_blocks(h, copies[:, 0], copies[:, 1])
        kv_append(h, 0, _dev(mix.k_new, device), _dev(mix.v_new, device), _dev(slots, device))
        q = _dev(mix.q, device)
        out = torch.empty((B, mix.Hq, mix.D), dtype=out_dtype, device=device)
        max_ctx = int(mix.ctx.max())
        _, _, ws = paged_decode_plan(B, mix.Hq, mix.Hkv, mix.D, max_ctx)
        workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=device)
        paged_decode_workspace_init(workspace)
        paged_decode_attention(q, k_pool[0], v_pool[0], _dev(table, device), _dev(mix.ctx, device), mix.scale, out,
                               workspace, max_ctx)
        torch.cuda.synchronize()
        return {"tables_before": tables_before, "block_table": table, "copies": copies, "slots": slots,
                "k_cache": k_pool[0], "v_cache": v_pool[0], "out": out, "handle": None}
    finally:
        kv_cache_destroy(h)


def prefill_then_decode(wl, causal=True, device="cuda", out_dtype=torch.float32, poison=True):
    """Prefill a packed batch, write all its K/V into a paged cache, then one decode token per sequence."""
    q, k, v = _dev(wl.q, device), _dev(wl.k, device), _dev(wl.v, device)
    cu = _dev(wl.cu_seqlens, device)
    T = q.shape[0]
    out = torch.empty((T, wl.Hq, wl.D), dtype=out_dtype, device=device)
    prefill_attention(q, k, v, cu, max(wl.seqlens), wl.scale, causal, out)
    n = len(wl.seqlens)
    cfg = KvcConfig(num_layers=1, num_blocks=wl.NB, num_kv_heads=wl.Hkv, head_dim=wl.D, block_size=wl.bs)
    alloc = poisoned_pool if poison else (lambda s, d: torch.zeros(s, dtype=torch.float16, device=d))
    k_pool, v_pool = alloc(cfg.pool_shape, device), alloc(cfg.pool_shape, device)
    h = kv_cache_create(cfg, k_pool, v_pool)
    try:
        seqlens = np.array(wl.seqlens, np.int32)
        slots = kv_slot_mapping(wl.block_table, np.zeros(n, np.int32), seqlens, wl.bs)
        kv_append(h, 0, k, v, _dev(slots, device))
        step = kv_slot_mapping(wl.block_table, seqlens, np.ones(n, np.int32), wl.bs)
        kv_append(h, 0, _dev(wl.k_dec, device), _dev(wl.v_dec, device), _dev(step, device))
        ctx = seqlens + 1
        dec = torch.empty((n, wl.Hq, wl.D), dtype=out_dtype, device=device)
        _, _, ws = paged_decode_plan(n, wl.Hq, wl.Hkv, wl.D, int(ctx.max()))
        workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=device)
        paged_decode_workspace_init(workspace)
        paged_decode_attention(_dev(wl.q_dec, device), k_pool[0], v_pool[0], _dev(wl.block_table, device),
                               _dev(ctx, device), wl.scale, dec, workspace, int(ctx.max()))
        torch.cuda.synchronize()
        return {"prefill_out": out, "decode_out": dec, "k_cache": k_pool[0], "v_cache": v_pool[0]}
    finally:
        kv_cache_destroy(h)


class TreeSession:
    """One step of tree-drafted decoding on a TreeWorkload: per layer kv_append_rope and paged_decode_tree_attention
    over the drafted nodes, then draft_tree_verify and kv_tree_commit.

    The step reads the sequences' lengths on the device only, and every call is prepared once, so it can be captured
    into a graph.  After it, `context_lens` (lengths with the drafted tree) is superseded by `new_context_lens` (with the
    kept path)."""

    def __init__(self, wl, device="cuda", out_dtype=torch.float16):
        self.wl, self.device = wl, device
        B, T, L, Hq, Hkv, D = len(wl.hist), wl.T, wl.L, wl.Hq, wl.Hkv, wl.D
        cfg = KvcConfig(num_layers=L, num_blocks=wl.NB, num_kv_heads=Hkv, head_dim=D, block_size=wl.bs)
        self.k_pool, self.v_pool = _dev(wl.k_pool, device), _dev(wl.v_pool, device)
        self.h = kv_cache_create(cfg, self.k_pool, self.v_pool)
        self.block_table, self.tree_lens = _dev(wl.block_table, device), _dev(wl.tree_lens, device)
        self.context_lens = _dev(wl.ctx, device)
        self.max_ctx = int(wl.block_table.shape[1]) * wl.bs
        masks, depths = kv_tree_masks(wl.parents, wl.tree_lens)
        self.masks = _dev(masks, device)
        self.positions = _dev((wl.hist[:, None] + depths).reshape(-1).astype(np.int32), device)
        slots = kv_slot_mapping(wl.block_table, wl.hist, np.full(B, T, np.int32), wl.bs).reshape(B, T)
        slots[np.arange(T)[None] >= wl.tree_lens[:, None]] = -1  # entries behind a tree are not appended
        self.slots = _dev(slots.reshape(-1), device)
        self.turns = _dev(kv_rope_turns(wl.inv_freq), device)
        self.qkv = _dev(wl.qkv, device)
        self.q_weight, self.k_weight = _dev(wl.q_weight, device), _dev(wl.k_weight, device)
        self.tokens, self.parents = _dev(wl.tokens, device), _dev(wl.parents, device)
        self.uniforms, self.p, self.q = _dev(wl.uniforms, device), _dev(wl.p, device), _dev(wl.q, device)
        self.q_rot = torch.zeros((L, B, T, Hq, D), dtype=torch.float16, device=device)
        self.out = torch.zeros((L, B, T, Hq, D), dtype=out_dtype, device=device)
        ws = paged_decode_tree_plan(B, Hq, Hkv, D, self.max_ctx, T)
        self.workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.path, self.path_len = torch.zeros((B, T), **i32), torch.zeros(B, **i32)
        self.next_token, self.new_context_lens = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self._calls = []
        for layer in range(L):
            q, k, v = (x.unflatten(1, (-1, D)) for x in self.qkv[layer].split((Hq * D, Hkv * D, Hkv * D), 1))
            self._calls.append(kv_append_rope(
                q, k, v, self.positions, self.turns, self.q_rot[layer].view(B * T, Hq, D), self.k_pool[layer],
                self.v_pool[layer], self.slots, q_weight=self.q_weight[layer], k_weight=self.k_weight[layer],
                eps=wl.eps, prepare=True))
            self._calls.append(paged_decode_tree_attention(
                self.q_rot[layer], self.k_pool[layer], self.v_pool[layer], self.block_table, self.context_lens,
                self.masks, wl.scale, self.out[layer], self.workspace, self.max_ctx, tree_lens=self.tree_lens,
                prepare=True))
        self._calls.append(draft_tree_verify(self.p, self.q, self.tokens, self.parents, self.uniforms, self.path,
                                             self.path_len, self.next_token, tree_lens=self.tree_lens, prepare=True))
        self._calls.append(kv_tree_commit(self.h, self.block_table, self.context_lens, self.path, self.path_len,
                                          self.new_context_lens, tree_lens=self.tree_lens, prepare=True))

    def step(self, stream=None):
        """The whole step on `stream` or the current one (asynchronous)."""
        if not self.h:
            raise ValueError("the session's cache was destroyed")
        for call in self._calls:
            call(stream)

    def close(self):
        if self.h:
            kv_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class ServingSession:
    """One layer of a serving loop whose request lengths stay on the GPU: prompts at once, then a token per sequence and
    step, over an fp16 cache or (block8) a block-scaled 8-bit one, with a sliding window and sinks or without.

    kv_block_tables places every step's tokens in blocks claimed from the library's pool (a windowed sequence goes
    through its own in turn), so a step reads nothing on the host and can be captured into a graph: its inputs are q, k
    and v, its output out."""

    def __init__(self, B, Hq, Hkv, D, num_blocks, max_len, window=0, sinks=0, block8=False, device="cuda",
                 out_dtype=torch.float16):
        self.window, self.sinks, self.max_len, self.scale = window, sinks, max_len, D ** -0.5
        f16, i32 = dict(dtype=torch.float16, device=device), dict(dtype=torch.int32, device=device)
        cfg = KvcConfig(num_layers=1, num_blocks=num_blocks, num_kv_heads=Hkv, head_dim=D)
        if block8:
            self.codes = torch.full((num_blocks, Hkv, 2, 16, D), 0x7f, dtype=torch.uint8, device=device)
            self.scales = torch.full((num_blocks, Hkv, 2), float("nan"), device=device)
            self.h = kv_cache_create(cfg)  # the block pool alone
        else:
            self.codes = None
            self.k_pool, self.v_pool = (poisoned_pool(cfg.pool_shape, device) for _ in range(2))
            self.h = kv_cache_create(cfg, self.k_pool, self.v_pool)
        self.free = torch.tensor([kv_block_alloc(self.h) for _ in range(num_blocks)], **i32)
        self.placed, self.new_placed = torch.zeros(1, **i32), torch.zeros(1, **i32)
        self.before, self.after = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.table = torch.full((B, -(-max_len // 16)), -1, **i32)
        self.cu, self.slots = torch.zeros(B + 1, **i32), torch.zeros(B, dtype=torch.int64, device=device)
        self.q, self.k, self.v = torch.zeros(B, Hq, D, **f16), torch.zeros(B, Hkv, D, **f16), torch.zeros(B, Hkv, D, **f16)
        self.out = torch.zeros(B, Hq, D, dtype=out_dtype, device=device)
        plan = paged_decode_fp8_block_plan if block8 else paged_decode_window_plan
        args = (B, Hq, Hkv, D, max_len)
        ws = plan(*args, window=window, sinks=sinks) if block8 or window else paged_decode_plan(*args)[2]
        self.workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=device)

    def _append(self, k, v, slots):
        if self.codes is not None:
            kv_append_fp8_block(k, v, slots, self.codes, self.scales)
        else:
            kv_append(self.h, 0, k, v, slots)

    def prompts(self, q, k, v, lens):
        """Attention of every sequence's prompt (packed, lens rows each) and its rows in the cache."""
        n = q.shape[0]
        self.after.copy_(torch.as_tensor(np.asarray(lens, np.int32)))
        slots = torch.zeros(n, dtype=torch.int64, device=q.device)
        out = torch.zeros(q.shape, dtype=self.out.dtype, device=q.device)
        kv_block_tables(None, self.after, self.free, self.placed, self.table, self.new_placed, self.cu, slots,
                        window=self.window, sinks=self.sinks)
        if self.window:
            prefill_window_attention(q, k, v, self.cu, max(lens), self.window, self.sinks, self.scale, out)
        else:
            prefill_attention(q, k, v, self.cu, max(lens), self.scale, True, out)
        self._append(k, v, slots)
        self.placed.copy_(self.new_placed)
        self.before.copy_(self.after)
        return out

    def step(self):
        """One token of every sequence, from self.q, self.k and self.v to self.out (asynchronous)."""
        torch.add(self.before, 1, out=self.after)
        kv_block_tables(self.before, self.after, self.free, self.placed, self.table, self.new_placed, self.cu, self.slots,
                        window=self.window, sinks=self.sinks)
        if self.codes is not None:
            self._append(self.k, self.v, self.slots)
        # (the copies also lie between the tables or the append and an attention launched with overlap)
        self.placed.copy_(self.new_placed)
        self.before.copy_(self.after)
        if self.codes is not None:
            paged_decode_attention_fp8_block(self.q, self.codes, self.scales, self.table, self.after, self.scale, self.out,
                                             self.workspace, self.max_len, window=self.window, sinks=self.sinks)
        elif self.window:
            paged_decode_window_attention(self.q, self.k_pool[0], self.v_pool[0], self.table, self.after, self.window,
                                          self.sinks, self.scale, self.out, self.workspace, self.max_len, k_new=self.k,
                                          v_new=self.v)
        else:
            paged_decode_append_attention(self.q, self.k, self.v, self.k_pool[0], self.v_pool[0], self.table, self.after,
                                          self.scale, self.out, self.workspace, self.max_len)

    def close(self):
        if self.h:
            kv_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _align16(n: int) -> int:
    return (n + 15) & ~15


class HostStep:
    """A DecodeSession's step fed from pinned host memory, its output returned there, with the copies overlapped
    with the calls as a serving loop whose inputs arrive from the host would run it.

    The step's inputs sit in one pinned host buffer: a header (block table, context lengths, append slots),
    then per layer that layer's q, k_new and v_new, each 16-byte aligned.  A device buffer has the same layout
    and every call receives views into it.  Every copy is a staging copy (kvc_copy_async: a kernel that reads or
    writes the pinned buffer over the host link) in the stream's kernel sequence.  In: the header with layers 0
    and 1 before layer 0's call; the later layers ahead, in pieces of growing size, each alongside an earlier
    layer's call (layers 2-3 alongside layer 0's, 4-7 alongside layer 1's, the rest alongside layer 3's; one
    piece for all of them made layer 1 wait for it).  Out: the outputs of layers
    [lo, hi) ahead, alongside layer hi's call (a decode call lets the next kernel start only once the calls before
    it have finished, so those outputs are final), eight layers at a time; the last layer's after its call.
    Every call is checked and converted once, at construction (the prepare=True form of the API)."""

    GROUP = 8  # layers per device-to-host copy

    def __init__(self, sess: DecodeSession):
        wl, dev = sess.wl, sess.device
        self.sess, self.device, self.L = sess, dev, wl.L
        parts = [("block_table", np.ascontiguousarray(wl.block_table, np.int32)),
                 ("context_lens", np.ascontiguousarray(wl.ctx, np.int32)),
                 ("slots", np.ascontiguousarray(sess.step_slots_host, np.int64))]
        for layer in range(wl.L):
            parts += [(("q", layer), np.ascontiguousarray(wl.q[layer], np.float16)),
                      (("k_new", layer), np.ascontiguousarray(wl.k_new[layer], np.float16)),
                      (("v_new", layer), np.ascontiguousarray(wl.v_new[layer], np.float16))]
        offs, pos, layer_end = {}, 0, []
        for name, a in parts:
            offs[name] = pos
            pos = _align16(pos + a.nbytes)
            if name[0] == "v_new":
                layer_end.append(pos)
        self.h_buf = torch.empty(pos, dtype=torch.uint8).pin_memory()
        hb = self.h_buf.numpy()
        hb[:] = 0
        for name, a in parts:
            hb[offs[name]:offs[name] + a.nbytes] = a.reshape(-1).view(np.uint8)
        self.d_buf = torch.zeros(pos, dtype=torch.uint8, device=dev)
        tdt = {np.dtype(np.int32): torch.int32, np.dtype(np.int64): torch.int64, np.dtype(np.float16): torch.float16}

        def view(name, a):
            return self.d_buf[offs[name]:offs[name] + a.nbytes].view(tdt[a.dtype]).view(a.shape)
        arrays = dict(parts)
        self.block_table, self.context_lens, self.slots = (view(n, arrays[n])
                                                          for n in ("block_table", "context_lens", "slots"))
        self.q, self.k_new, self.v_new = ([view((n, layer), arrays[(n, layer)]) for layer in range(wl.L)]
                                          for n in ("q", "k_new", "v_new"))
        self.k_pool = [sess.k_pool[layer] for layer in range(wl.L)]
        self.v_pool = [sess.v_pool[layer] for layer in range(wl.L)]
        self.out = [sess.out[layer] for layer in range(wl.L)]
        self.h_out = torch.empty(sess.out.shape, dtype=sess.out.dtype).pin_memory()
        self.h_out_layers = [self.h_out[layer] for layer in range(wl.L)]
        cut = layer_end[min(1, wl.L - 1)]  # header + layers 0 and 1
        self.first = (self.d_buf[:cut], self.h_buf[:cut])
        # layers [a, b) staged ahead alongside layer a / 2 - 1's call
        starts = [a for a in (2, 4, 8) if a < wl.L]
        self.ahead_in = {}
        for i, a in enumerate(starts):
            b = starts[i + 1] if i + 1 < len(starts) else wl.L
            lo, hi = layer_end[a - 1], layer_end[b - 1]
            self.ahead_in[a // 2 - 1] = (self.d_buf[lo:hi], self.h_buf[lo:hi])
        # device-to-host groups [lo, hi) of all layers but the last, each sent alongside layer hi's call
        self.groups = {min(g + self.GROUP, wl.L - 1): (self.h_out[g:min(g + self.GROUP, wl.L - 1)],
                                                       sess.out[g:min(g + self.GROUP, wl.L - 1)])
                       for g in range(0, wl.L - 1, self.GROUP)}
        self.h2d_bytes = pos
        self.d2h_bytes = self.h_out.numel() * self.h_out.element_size()
        # every call of the step checked and converted once (PreparedCall); run() only launches them
        self._first = kvc_copy_async(*self.first, prepare=True)
        self._ahead_in = {k: kvc_copy_async(*v, ahead=True, prepare=True) for k, v in self.ahead_in.items()}
        self._groups = {k: kvc_copy_async(*v, ahead=True, prepare=True) for k, v in self.groups.items()}
        self._last = kvc_copy_async(self.h_out_layers[-1], self.out[-1], prepare=True)
        self._fused = [paged_decode_append_attention(self.q[layer], self.k_new[layer], self.v_new[layer],
                                                     self.k_pool[layer], self.v_pool[layer], self.block_table,
                                                     self.context_lens, wl.scale, self.out[layer], sess.workspace,
                                                     sess.max_ctx, sess.blocks_per_split, prepare=True)
                       for layer in range(wl.L)]
        self._unfused = [(kv_append(sess.h, layer, self.k_new[layer], self.v_new[layer], self.slots, prepare=True),
                          paged_decode_attention(self.q[layer], self.k_pool[layer], self.v_pool[layer],
                                                 self.block_table, self.context_lens, wl.scale, self.out[layer],
                                                 sess.workspace, sess.max_ctx, sess.blocks_per_split, prepare=True))
                         for layer in range(wl.L)]

    def run(self, fused=True):
        """One step on the current stream: copies in, every layer's call(s), copies out (all asynchronous)."""
        cs = torch.cuda.current_stream(self.device)
        self._first(cs)
        for layer in range(self.L):
            if fused:
                self._fused[layer](cs)
            else:
                append, decode = self._unfused[layer]
                append(cs)
                decode(cs)
            if layer in self._ahead_in:
                self._ahead_in[layer](cs)
            if layer in self._groups:
                self._groups[layer](cs)
        self._last(cs)
