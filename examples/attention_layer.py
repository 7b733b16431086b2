"""One attention layer of multi-adapter serving, from its input rows to its
output rows, with every step in the library:

  qkv   = Wqkv x + B_s A_s x          lora_base_gemm_apply (adapter s of the row),
                                      lora_base_q4_apply where W is kept in 4 bits
  q, k  = rotate(norm(q)), rotate(norm(k)); k and v into their pages
                                      lora_rope_append
  attn  = softmax(q K^T) V            lora_paged_attention
  y     = Wo attn + B_s A_s attn      as qkv

A tree of drafted tokens goes through the same layer in one step: each token's
position is the context's length plus its depth, lora_tree_attention lets it see
its own branch, and lora_kv_keep_rows moves the accepted branch's rows up.

Sequences are appended to, forked (sharing pages, copied on write), ended and
compacted with lk.Pages and lora_kv_copy_pages.  Run as a program it decodes a
few requests and verifies drafted tokens on random weights:

    python -m examples.attention_layer
"""
from __future__ import annotations

import numpy as np
import torch

import adapter_sgmv_lora_gb300 as lk


def quantize(w, group_size):
    """w [out, in] in 4 bits, to the nearest: codes 1..15 around a zero of 8, a scale for each group of inputs."""
    out, n = w.shape
    groups = -(-n // group_size)
    pad = torch.nn.functional.pad(w.float(), (0, groups * group_size - n)).unflatten(1, (groups, group_size))
    scales = (pad.abs().amax(-1) / 7).clamp_min(1e-12).to(w.dtype)
    codes = (torch.round(pad / scales.float().unsqueeze(-1)).clamp(-7, 7) + 8).flatten(1)[:, :n].to(torch.uint8)
    codes = torch.nn.functional.pad(codes, (0, n % 2))
    return lk.Q4Weight((codes[:, ::2] | codes[:, 1::2] << 4).contiguous(), scales, group_size)


class AttentionLayer:
    """The layer with its adapters, cache and sequences.  Sequence s runs on
    adapter slot `adapter[s]` (-1: the base model).  group_size: keep the
    projections in 4 bits, in groups of so many inputs."""

    def __init__(self, hidden, heads, kv_heads, head_dim, max_loras, max_rank, num_pages, page_size, max_seqs,
                 max_pages, dtype=torch.bfloat16, theta=500000.0, seed=0, device="cuda", group_size=None):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *shape, scale: (torch.randn(shape, generator=g) * scale).to(dtype).to(device)
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.dtype = hidden, heads, kv_heads, head_dim, dtype
        self.max_loras, self.device = max_loras, device
        self.qkv_dims = [heads * head_dim, kv_heads * head_dim, kv_heads * head_dim]
        self.w_qkv = [rand(o, hidden, scale=hidden ** -0.5) for o in self.qkv_dims]
        self.w_o = [rand(hidden, heads * head_dim, scale=(heads * head_dim) ** -0.5)]
        if group_size is not None:
            self.w_qkv, self.w_o = ([quantize(w, group_size) for w in ws] for ws in (self.w_qkv, self.w_o))
        self.q_norm, self.k_norm = rand(head_dim, scale=0.1) + 1, rand(head_dim, scale=0.1) + 1
        # per-slot stacks, zero until an adapter is loaded
        z = lambda *shape: torch.zeros(shape, dtype=dtype, device=device)
        self.a_qkv, self.b_qkv = z(max_loras, 3 * max_rank, hidden), z(max_loras, sum(self.qkv_dims), max_rank)
        self.a_o, self.b_o = z(max_loras, max_rank, heads * head_dim), z(max_loras, hidden, max_rank)
        self.rope = lk.rope_to_device(lk.lora_build_rope(head_dim, theta), device)
        pool = lambda: torch.zeros((num_pages, page_size, kv_heads, head_dim), dtype=dtype, device=device)
        self.cache = lk.KVCache(pool(), pool())
        self.caches = lk.KVCaches([self.cache])  # a model lists its layers here
        self.pages = lk.Pages(num_pages, page_size, max_seqs, max_pages)
        self.adapter = np.full(max_seqs, -1, dtype=np.int32)
        self.drafts = {}  # drafted tokens that verify left for keep, of each sequence

    def load_adapter(self, slot, rank, alpha, a_qkv, b_qkv, a_o, b_o):
        """Raw fp32 adapter: a_qkv[j] [rank, hidden], b_qkv[j] [out_j, rank] for q, k, v; a_o, b_o."""
        x = torch.empty((1, self.hidden), dtype=self.dtype, device=self.device)
        y = torch.empty((1, sum(self.qkv_dims)), dtype=self.dtype, device=self.device)
        p = lk.fused_problem(x, self.a_qkv, self.b_qkv, y, self.qkv_dims)
        for j in range(3):
            lk.lora_set_slot(p, j, slot, rank, alpha, False, a_qkv[j], b_qkv[j])
        x = torch.empty((1, self.heads * self.head_dim), dtype=self.dtype, device=self.device)
        y = torch.empty((1, self.hidden), dtype=self.dtype, device=self.device)
        lk.lora_set_slot(lk.fused_problem(x, self.a_o, self.b_o, y, [self.hidden]), 0, slot, rank, alpha, False,
                         a_o, b_o)

    def _project(self, x, a, b, out_dims, weights, route):
        y = torch.empty((x.shape[0], sum(out_dims)), dtype=self.dtype, device=self.device)
        p = lk.fused_problem(x, a, b, y, out_dims)
        routing, workspace = lk.routing_to_device(route, self.device), lk.new_workspace(p, route["end"], self.device)
        if isinstance(weights[0], lk.Q4Weight):
            lk.lora_base_q4_apply(lk.BaseQ4Problem(p, routing, weights), workspace)
        else:
            lk.lora_base_gemm_apply(p, routing, weights, workspace)
        return y

    def _settled(self, seqs):
        for s in seqs:
            if s in self.drafts:
                raise ValueError("sequence %d has drafted tokens: keep says first which of them stay" % s)

    def _append(self, seqs, counts, depths=None):
        """Rows and positions (depths[i] behind the sequence's end; None: one after the other) of counts[i] more
        tokens of seqs[i]; runs the copies that shared pages need.  Where the pages do not suffice for all of them
        the sequences stay as long as they were."""
        rows, positions, copies, starts = [], [], [], []
        try:
            for i, (s, n) in enumerate(zip(seqs, counts)):
                start = int(self.pages.lengths[s])
                r, c = self.pages.append(s, n)
                starts.append(start)
                rows.append(r)
                copies += c
                positions.append(start + (np.arange(n) if depths is None else depths[i]))
        except lk.LoraError:
            for s, start in reversed(list(zip(seqs, starts))):
                self.pages.trim(s, start)
            raise
        finally:  # the tables name the copies already, on an error too
            if copies:
                lk.lora_kv_copy_pages(self.caches, *zip(*copies))
        up = lambda a: torch.from_numpy(np.concatenate(a).astype(np.int32)).to(self.device)
        return up(rows), up(positions)

    def _store(self, x, seqs, counts, route, depths=None):
        """qkv of sorted rows, rotated; k and v into the cache.  Returns the rotated queries [T, heads, hd]."""
        H, Hk, hd = self.heads, self.kv_heads, self.head_dim
        self._settled(seqs)
        rows, positions = self._append(seqs, counts, depths)
        y = self._project(x, self.a_qkv, self.b_qkv, self.qkv_dims, self.w_qkv, route)
        q, k, v = (y[:, a:b].unflatten(1, (-1, hd)) for a, b in ((0, H * hd), (H * hd, (H + Hk) * hd),
                                                                 ((H + Hk) * hd, (H + 2 * Hk) * hd)))
        lk.lora_rope_append(lk.RopeProblem(q=q, k=k, v=v, q_out=q, rope=self.rope, positions=positions,
                                           cache=self.cache, cache_rows=rows, q_weight=self.q_norm,
                                           k_weight=self.k_norm))
        return q

    def prefill(self, seqs, xs):
        """Store the tokens xs[i] [n_i, hidden] of each sequence (no output: a prompt's last token is decoded)."""
        counts = [x.shape[0] for x in xs]
        route = lk.lora_build_routing(self.adapter[seqs], counts, self.max_loras)
        order = route["perm"]
        self._store(torch.cat([xs[i] for i in order]), [seqs[i] for i in order], [counts[i] for i in order], route)

    def decode(self, seqs, x):
        """One token x[i] of each sequence; returns y [len(seqs), hidden] in the same order."""
        route = lk.lora_build_routing(self.adapter[seqs], [1] * len(seqs), self.max_loras)
        order = route["perm"].astype(np.int64)
        mine = [seqs[i] for i in order]
        pick = torch.from_numpy(order).to(self.device)
        q = self._store(x[pick], mine, [1] * len(mine), route)
        attn = torch.empty((len(mine), self.heads, self.head_dim), dtype=self.dtype, device=self.device)
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(self.device)
        # q is the q part of the fused rows: attention takes it where it is
        problem = lk.AttentionProblem(q=q, out=attn, cache=self.cache, block_tables=up(self.pages.tables[mine]),
                                      lengths=up(self.pages.lengths[mine]))
        lk.lora_paged_attention(problem, lk.new_attention_workspace(problem))
        y = self._project(attn.flatten(1), self.a_o, self.b_o, [self.hidden], self.w_o, route)
        out = torch.empty_like(y)
        out[pick] = y
        return out

    def verify(self, seqs, xs, parents):
        """A tree of drafted tokens of each sequence: token j of seqs[i] is xs[i][j] and follows drafted token
        parents[i][j] (-1: the cached context).  Returns the output rows [n_i, hidden] of each sequence, whose
        rows stay in the cache until keep says which branch was accepted; until then it takes no other tokens and is
        not forked."""
        counts = [x.shape[0] for x in xs]
        route = lk.lora_build_routing(self.adapter[seqs], counts, self.max_loras)
        order = [int(i) for i in route["perm"]]
        mine, n = [seqs[i] for i in order], [counts[i] for i in order]
        words = max(1, -(-max(counts) // 64))
        trees = [lk.lora_build_tree(parents[i], words) for i in order]
        q = self._store(torch.cat([xs[i] for i in order]), mine, n, route, [t["depths"] for t in trees])
        attn = torch.empty((sum(n), self.heads, self.head_dim), dtype=self.dtype, device=self.device)
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(self.device)
        offsets = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
        problem = lk.TreeAttentionProblem(q=q, out=attn, cache=self.cache, block_tables=up(self.pages.tables[mine]),
                                          lengths=up(self.pages.lengths[mine]), row_offsets=up(offsets),
                                          masks=up(np.concatenate([t["masks"] for t in trees]).view(np.int64)))
        lk.lora_tree_attention(problem, lk.new_tree_attention_workspace(problem))
        y = self._project(attn.flatten(1), self.a_o, self.b_o, [self.hidden], self.w_o, route)
        self.drafts.update(zip(mine, n))
        rows = {s: y[a:b] for s, a, b in zip(mine, offsets, offsets[1:])}
        return [rows[s] for s in seqs]

    def keep(self, paths):
        """Of the drafted tokens that verify left keep paths[seq], a branch from its root on; a sequence that is not
        named keeps none."""
        mine, n = list(self.drafts), list(self.drafts.values())
        self.drafts = {}
        if not mine:
            return
        kept = [list(paths.get(s, [])) for s in mine]
        path = np.full((len(mine), max(map(len, kept))), -1, dtype=np.int32)
        for row, k in zip(path, kept):
            row[:len(k)] = k
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(self.device)
        # the pages as they are now: compact may have moved them
        lk.lora_kv_keep_rows(lk.KeepRowsProblem(self.caches, up(self.pages.tables[mine]), up(self.pages.lengths[mine]),
                                                up(np.cumsum([0] + n)), up(path)))
        for s, rows, k in zip(mine, n, kept):
            self.pages.trim(s, int(self.pages.lengths[s]) - rows + len(k))

    def fork(self, parent, child):
        self._settled([parent])
        self.pages.fork(parent, child)
        self.adapter[child] = self.adapter[parent]

    def end(self, seq):
        self.drafts.pop(seq, None)
        self.pages.trim(seq, 0)
        self.adapter[seq] = -1

    def compact(self):
        src, dst = self.pages.compact()
        lk.lora_kv_copy_pages(self.caches, src, dst)
        return len(src)


def demo_layer(seed=0, **kw):
    """A small layer with three adapters loaded."""
    size = dict(hidden=256, heads=8, kv_heads=2, head_dim=64, max_loras=3, max_rank=16, num_pages=64, page_size=16,
                max_seqs=8, max_pages=16)
    layer = AttentionLayer(**{**size, **kw}, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    rand = lambda *shape, scale: (torch.randn(shape, generator=g) * scale).cuda()
    layer.raw = []
    for slot, rank in enumerate((8, 16, 4)):
        n = layer.heads * layer.head_dim
        raw = dict(rank=rank, alpha=2.0 * rank,
                   a_qkv=[rand(rank, layer.hidden, scale=layer.hidden ** -0.5) for _ in range(3)],
                   b_qkv=[rand(o, rank, scale=0.1) for o in layer.qkv_dims], a_o=rand(rank, n, scale=n ** -0.5),
                   b_o=rand(layer.hidden, rank, scale=0.1))
        layer.raw.append(raw)
        layer.load_adapter(slot, **raw)
    return layer


def verify_drafts():
    """Two requests on 4-bit weights: prompts, a tree of drafted tokens for each, the accepted branches, a step on."""
    layer = demo_layer(group_size=64)
    x = lambda n: torch.randn((n, layer.hidden), device="cuda").to(layer.dtype)
    layer.adapter[[0, 1]] = [2, -1]
    layer.prefill([0, 1], [x(30), x(7)])
    trees = [[-1, 0, 0, 1, 1, 2], [-1, 0, 1]]     # a tree of six and a chain of three
    ys = layer.verify([0, 1], [x(len(t)) for t in trees], trees)
    layer.keep({0: [0, 2, 5], 1: [0]})
    layer.decode([0, 1], x(2))
    assert lk.lora_get_device_status() == 0
    print("verified %s drafted tokens; lengths %s" % ([len(y) for y in ys], layer.pages.lengths[:2].tolist()))


def main():
    verify_drafts()
    layer = demo_layer()
    rng = np.random.default_rng(0)
    x = lambda n: torch.randn((n, layer.hidden), device="cuda").to(layer.dtype)
    seqs = [0, 1, 2, 3]
    layer.adapter[seqs] = [1, 0, -1, 2]
    layer.prefill(seqs, [x(int(n)) for n in rng.integers(5, 100, size=4)])
    layer.fork(0, 4)                              # two continuations of one prompt
    for _ in range(8):
        layer.decode([0, 1, 2, 3, 4], x(5))
    layer.end(1)
    moved = layer.compact()
    y = layer.decode([0, 2, 3, 4], x(4))
    assert lk.lora_get_device_status() == 0
    print("decoded %s rows; lengths %s; %d pages in use after a compaction that moved %d" %
          (tuple(y.shape), layer.pages.lengths[:5].tolist(), int((layer.pages.refs > 0).sum()), moved))


if __name__ == "__main__":
    main()
