"""The step that verifies drafted tokens on a 4-bit base model, and its plain forms.

A served model that drafts tokens ahead checks them in one pass over few rows:
a tree (or a chain) of drafted tokens per sequence goes through the projections,
its keys and values are appended to the paged cache, every drafted token
attends to the sequence's context and to its own branch, and the rows of the
accepted branch are kept.  Three operators do that:

  q4    lora_base_q4_apply: the base projection with 4-bit weights and group
        scales, the LoRA delta of each row's adapter joined before the rounding
  tree  lora_tree_attention: drafted tokens over the paged cache, each seeing
        the context and the drafted tokens that its mask names
  keep  lora_kv_keep_rows: the accepted branch's cache rows moved up behind
        the context, in every layer

`own` False runs each in elementary torch operations in 32 bits, rounded once
at the end; True makes the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases --

def _q4(name, in_dim, outs, seqs, min_rows, max_rows, group, rank, slots, base=0.2, zeros=False, dtype="bf16", pad=0,
        shape_seed=1):
    return dict(name=name, op="q4", in_dim=in_dim, out0=outs[0], out1=outs[1] if len(outs) > 1 else 0,
                out2=outs[2] if len(outs) > 2 else 0, seqs=seqs, min_rows=min_rows, max_rows=max_rows, group=group,
                rank=rank, slots=slots, base=base, zeros=zeros, dtype=dtype, pad=pad, shape_seed=shape_seed)


def _tree(name, seqs, min_rows, max_rows, min_ctx, max_ctx, heads, kv_heads, head_dim, dtype="bf16", page_size=16,
          order="token", chain=False, empty=0, pad=0, lse=False, shape_seed=1):
    return dict(name=name, op="tree", seqs=seqs, min_rows=min_rows, max_rows=max_rows, min_ctx=min_ctx,
                max_ctx=max_ctx, heads=heads, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype, page_size=page_size,
                order=order, chain=chain, empty=empty, pad=pad, lse=lse, shape_seed=shape_seed)


def _keep(name, layers, seqs, min_rows, max_rows, min_ctx, max_ctx, kept, kv_heads, head_dim, dtype="bf16",
          page_size=16, order="token", shape_seed=1):
    return dict(name=name, op="keep", layers=layers, seqs=seqs, min_rows=min_rows, max_rows=max_rows,
                min_ctx=min_ctx, max_ctx=max_ctx, kept=kept, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype,
                page_size=page_size, order=order, shape_seed=shape_seed)


def listed():
    return [
        # one token of one request on the 8B qkv projection: latency and the weights alone
        _q4("q4_qkv8b_1", 4096, [4096, 1024, 1024], 1, 1, 1, 128, 16, 8, base=0.0),
        # a chain of five drafted tokens of one request on the 8B gate and up projections, zero points, small groups
        _q4("q4_gateup8b_5", 4096, [14336, 14336], 1, 5, 5, 64, 16, 8, base=0.0, zeros=True),
        # eight one-token requests and short chains, several adapters and base rows, on the 8B o_proj
        _q4("q4_o8b_29", 4096, [4096], 13, 1, 4, 128, 16, 8),
        # the trees of eight requests on the 70B qkv projection, rank 64
        _q4("q4_qkv70b_trees", 8192, [8192, 1024, 1024], 8, 9, 26, 128, 64, 8),
        # fp32, odd widths, a group that does not divide the row
        _q4("q4_f32_odd", 1013, [777, 130], 3, 1, 3, 40, 8, 3, zeros=True, dtype="f32"),
        # a chain of six drafted tokens of one request with a short context: latency alone
        _tree("tree_chain_1x6", 1, 6, 6, 517, 517, 32, 8, 128, chain=True),
        # a decode batch of 48 requests, ragged trees over ragged contexts on the 8B attention
        _tree("tree_48_8b", 48, 5, 26, 128, 2048, 32, 8, 128, pad=7),
        # one request with a long context and a wide tree: the split over its length alone fills the GPU
        _tree("tree_1x60_131072", 1, 60, 60, 131012, 131012, 32, 8, 128, page_size=32, lse=True),
        # trees of 64 on the 70B attention (8 query heads share a key/value head): the tensor cores' case
        _tree("tree_24x64_70b", 24, 64, 64, 1024, 8192, 64, 8, 128, page_size=64, order="head"),
        # fp32, odd sizes, sequences without a context whose first row sees nothing
        _tree("tree_f32_ragged", 19, 1, 13, 1, 901, 12, 4, 80, dtype="f32", page_size=8, empty=2, lse=True),
        # one request's accepted branch, all layers of an 8B model: latency alone
        _keep("keep_1", 32, 1, 26, 26, 517, 517, 4, 8, 128),
        # a batch of 64 requests, all layers of an 8B model
        _keep("keep_64", 32, 64, 8, 40, 20, 150, 7, 8, 128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["q4", "q4", "tree", "tree", "keep"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    group = rng.choice([1, 3, 4, 4, 7, 8, 8, 16])
    heads = kv_heads * min(group, max(1, 64 // kv_heads))
    head_dim = rng.choice([32, 64, 80, 96, 128, 128, 128, 256])
    page_size = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    order = rng.choice(["token", "head"])
    seed = rng.randrange(1 << 30)
    if op == "q4":
        big = 8192 * 10240 if dtype == "bf16" else 2048 * 2048
        in_dim = _log_int(rng, 64, 8192)
        in_dim = in_dim if rng.random() < 0.2 else -(-in_dim // 64) * 64
        n = rng.choice([1, 2, 3])
        outs = [_log_int(rng, 16, max(16, min(14336, big // in_dim // n))) for _ in range(n)]
        outs = outs if rng.random() < 0.2 else [-(-o // 16) * 16 for o in outs]
        rows = _log_int(rng, 1, 160 if dtype == "bf16" else 16)
        seqs = _log_int(rng, 1, min(rows, 24))
        most = max(1, rows // seqs)
        c = _q4(None, in_dim, outs, seqs, max(1, most // rng.choice([1, 2, 4])), most,
                rng.choice([32, 64, 64, 128, 128, 256, in_dim]), rng.choice([8, 16, 16, 32, 64, 128]),
                rng.choice([1, 4, 8, 16]), base=rng.choice([0.0, 0.2, 1.0]), zeros=rng.random() < 0.5, dtype=dtype,
                pad=rng.choice([0, 0, 3]), shape_seed=seed)
    elif op == "tree":
        budget = 24 * 4600 * 8 * 128 * 2            # cache elements of the largest listed case, K and V each
        most = budget // 2 // (kv_heads * head_dim * BYTES[dtype])
        seqs = _log_int(rng, 1, 100)
        work = 24 * 64 * 64 * 4600 // (1 if dtype == "bf16" else 32)  # rows x heads x context of that case
        ctx = _log_int(rng, 1, max(1, min(131072, most // seqs)))
        rows = _log_int(rng, 1, max(1, min(128, work // (seqs * heads * ctx), 2 ** 19 // (seqs * heads))))
        empty = rng.choice([0, 0, 1, 2]) if seqs > 3 else 0
        c = _tree(None, seqs, max(1, rows // rng.choice([1, 2, 8])), rows, max(1, ctx // rng.choice([1, 2, 16])), ctx,
                  heads, kv_heads, head_dim, dtype=dtype, page_size=page_size, order=order, chain=rng.random() < 0.3,
                  empty=empty, pad=rng.choice([0, 0, 5]), lse=rng.random() < 0.5, shape_seed=seed)
        if c["chain"]:
            c["empty"] = 0
    else:
        token = kv_heads * head_dim * BYTES[dtype]
        layers = _log_int(rng, 1, 64)
        seqs = _log_int(rng, 1, max(1, min(200, 2 ** 29 // (layers * token * 300))))
        rows = _log_int(rng, 1, 64)
        ctx = _log_int(rng, 1, 150)
        c = _keep(None, layers, seqs, max(1, rows // 4), rows, max(1, ctx // 8), ctx, rng.choice([1, 3, 6, 12]),
                  kv_heads, head_dim, dtype=dtype, page_size=page_size, order=order, shape_seed=seed)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype, scale=1.0):
    """N(0, scale^2), made in the type itself."""
    t = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return t.mul_(scale) if scale != 1.0 else t


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _outs(case):
    return [o for o in (case["out0"], case["out1"], case["out2"]) if o]


def _routes(case):
    """(slot of each group, first row of each group and the end, all rows): sequences sorted by adapter, base last."""
    r = random.Random(case["shape_seed"])
    counts = [r.randint(case["min_rows"], case["max_rows"]) for _ in range(case["seqs"])]
    slots = [-1 if r.random() < case["base"] else r.randrange(case["slots"]) for _ in counts]
    ids = sorted({s for s in slots if s >= 0})
    offs = [0]
    for s in ids:
        offs.append(offs[-1] + sum(n for n, t in zip(counts, slots) if t == s))
    return ids, offs, sum(counts) + case["pad"]


def _q4_data(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    n, outs = case["in_dim"], _outs(case)
    O, groups, R, S = sum(outs), -(-n // case["group"]), case["rank"], case["slots"]
    ids, offs, T = _routes(case)
    q = torch.randint(0, 256, (O, -(-n // 2)), generator=g, device="cuda", dtype=torch.uint8)
    # weights of variance about 1 / in_dim: codes less their zero have a deviation of 4.6
    scales = (torch.rand((O, groups), generator=g, device="cuda") + 0.5).mul_(1 / (4.6 * math.sqrt(n))).to(dt)
    zeros = torch.randint(5, 11, (O, groups), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    a = _randn((S, len(outs) * R, n), g, dt, 1 / math.sqrt(n))
    b = _randn((S, O, R), g, dt, 0.1)
    x = _randn((T, n), g, dt)
    return dict(q=q, scales=scales, zeros=zeros, a=a, b=b, x=x, ids=ids, offs=offs, T=T, outs=outs)


def _shapes(case):
    """Drafted rows and context of each sequence, the parent of each drafted token (-1: the context's end), and
    which sequences start with a row that sees nothing."""
    r = random.Random(case["shape_seed"])
    rows = [r.randint(case["min_rows"], case["max_rows"]) for _ in range(case["seqs"])]
    ctx = [r.randint(case["min_ctx"], case["max_ctx"]) for _ in rows]
    parents = [[-1] + [r.randrange(max(0, i - 9), i) for i in range(1, n)] for n in rows]
    blind = set(r.sample(range(len(rows)), case.get("empty", 0)))
    return rows, [0 if b in blind else c for b, c in enumerate(ctx)], parents, blind


def _masks(parents, blind, words):
    masks = np.zeros((sum(len(p) for p in parents), words), dtype=np.uint64)
    at = 0
    for b, par in enumerate(parents):
        seen = []
        for i, p in enumerate(par):
            seen.append((seen[p] if p >= 0 else 0) | (1 << i))
        for i, m in enumerate(seen):
            m = m & ~1 if b in blind else m         # nothing sees the first token, not even itself
            masks[at + i] = [(m >> (64 * w)) & (2 ** 64 - 1) for w in range(words)]
        at += len(par)
    return masks


def _tables(lens, page_size, r):
    need = [-(-n // page_size) for n in lens]
    num_pages = sum(need) + 3
    ids = list(range(num_pages))
    r.shuffle(ids)
    tables = np.full((len(lens), max(1, max(need))), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
    return tables, num_pages


def _pool(case, shape, g):
    """Pages as [..., pages, page_size, kv_heads, head_dim] views of token-major or head-major memory."""
    ps, h, d, dt = case["page_size"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    t = _randn(shape + ((ps, h, d) if case["order"] == "token" else (h, ps, d)), g, dt)
    return t if case["order"] == "token" else t.transpose(-2, -3)


def _tree_data(case, seed):
    g = _gen(seed)
    r = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    rows, ctx, parents, blind = _shapes(case)
    lens = [c + n for c, n in zip(ctx, rows)]
    tables, num_pages = _tables(lens, case["page_size"], r)
    n = sum(rows)
    masks = None
    if not case["chain"]:
        words = -(-max(rows) // 64)
        masks = torch.from_numpy(_masks(parents, blind, words).view(np.int64)).cuda()
    q = _randn((n + case["pad"], case["heads"], case["head_dim"]), g, dt, 1.5)
    return dict(q=q, kc=_pool(case, (num_pages,), g), vc=_pool(case, (num_pages,), g), tables=_ints(tables),
                lengths=_ints(lens), offsets=_ints(np.cumsum([0] + rows)), masks=masks, rows=rows, ctx=ctx, n=n,
                scale=1.0 / math.sqrt(case["head_dim"]))


def _keep_data(case, seed):
    g = _gen(seed)
    r = random.Random(seed)
    rows, ctx, _, _ = _shapes(case)
    lens = [c + n for c, n in zip(ctx, rows)]
    tables, num_pages = _tables(lens, case["page_size"], r)
    path = np.full((len(rows), case["kept"]), -1, dtype=np.int32)
    for b, n in enumerate(rows):
        m = min(n, r.randint(0, case["kept"]))
        path[b, :m] = sorted(r.sample(range(n), m))
    # every layer's K and V in one allocation, a layer's pools are views of it
    pools = _pool(case, (case["layers"], 2, num_pages), g)
    return dict(pools=pools, tables=_ints(tables), lengths=_ints(lens), offsets=_ints(np.cumsum([0] + rows)),
                path=_ints(path), new_lengths=_ints(np.zeros(len(rows))))


def prepare(case, seed):
    if case["op"] == "q4":
        s = _q4_data(case, seed)
        s["y"] = torch.zeros((s["T"], sum(s["outs"])), device="cuda", dtype=s["x"].dtype)
        s["offsets"], s["slots"] = _ints(s["offs"]), _ints(s["ids"])
        if own:
            import adapter_sgmv_lora_gb300 as lk
            cut = np.cumsum([0] + s["outs"])
            weights = [lk.Q4Weight(s["q"][i:j], s["scales"][i:j], case["group"],
                                   zeros=None if s["zeros"] is None else s["zeros"][i:j])
                       for i, j in zip(cut[:-1], cut[1:])]
            problem = lk.fused_problem(s["x"], s["a"], s["b"], s["y"], s["outs"])
            routing = lk.Routing(s["slots"], s["offsets"], len(s["ids"]), s["offs"][-1],
                                 host_grouped_offsets=np.array(s["offs"], dtype=np.int32),
                                 host_lora_ids=np.array(s["ids"], dtype=np.int32))
            s["problem"] = lk.BaseQ4Problem(problem, routing, weights)
            s["workspace"] = lk.new_workspace(problem, s["offs"][-1])
    elif case["op"] == "tree":
        s = _tree_data(case, seed)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(s["q"].shape[:2], device="cuda") if case["lse"] else None
        if own:
            import adapter_sgmv_lora_gb300 as lk
            if s["masks"] is not None and case["pad"]:   # the library wants a mask row for each row of q
                s["masks"] = torch.nn.functional.pad(s["masks"], (0, 0, 0, case["pad"]))
            s["problem"] = lk.TreeAttentionProblem(q=s["q"], out=s["out"], cache=lk.KVCache(s["kc"], s["vc"]),
                                                   block_tables=s["tables"], lengths=s["lengths"],
                                                   row_offsets=s["offsets"], masks=s["masks"], scale=s["scale"],
                                                   lse=s["lse"])
            s["workspace"] = lk.new_tree_attention_workspace(s["problem"])
    else:
        s = _keep_data(case, seed)
        if own:
            import adapter_sgmv_lora_gb300 as lk
            caches = lk.KVCaches([lk.KVCache(p[0], p[1]) for p in s["pools"]])
            s["problem"] = lk.KeepRowsProblem(caches=caches, block_tables=s["tables"], lengths=s["lengths"],
                                              row_offsets=s["offsets"], path=s["path"],
                                              new_lengths=s["new_lengths"])
    s["case"] = case
    return s


# ------------------------------------------------------------ plain forms --

def _plain_q4(s):
    case = s["case"]
    n, R, S, outs = case["in_dim"], case["rank"], case["slots"], s["outs"]
    codes = torch.stack((s["q"] & 15, s["q"] >> 4), -1).flatten(1)[:, :n].float()
    of = torch.arange(n, device="cuda") // case["group"]
    zero = 8.0 if s["zeros"] is None else s["zeros"].float()[:, of]
    w = (codes - zero) * s["scales"].float()[:, of]
    x = s["x"].float()
    y = x @ w.T
    if s["ids"]:
        # each routed row's own slot's block of A x, zero in the others', against all slots' B
        row = torch.arange(s["T"], device="cuda")
        group = torch.bucketize(row, s["offsets"][1:].long(), right=True).clamp(max=len(s["ids"]) - 1)
        mine = (torch.arange(S, device="cuda")[None, :] == s["slots"][group][:, None]) & (row < s["offs"][-1])[:, None]
        u = (x @ s["a"].float().flatten(0, 1).T).view(s["T"], S, len(outs), R) * mine[:, :, None, None]
        b = s["b"].float().split(outs, 1)
        y = y + torch.cat([torch.einsum("tsr,sor->to", u[:, :, j], b[j]) for j in range(len(outs))], 1)
    s["y"].copy_(y)
    return s["y"]


def _plain_tree(s):
    case = s["case"]
    B, hk, d, n, m = case["seqs"], case["kv_heads"], case["head_dim"], s["n"], max(s["rows"])
    G = case["heads"] // hk
    tables = s["tables"].clamp(min=0).long()
    k = s["kc"][tables].flatten(1, 2).float()                     # [B, L, hk, d]
    v = s["vc"][tables].flatten(1, 2).float()
    at = torch.arange(n, device="cuda")
    seq = torch.bucketize(at, s["offsets"][1:].long(), right=True)
    i = at - s["offsets"][seq].long()                             # a row's number within its sequence
    ctx = (s["lengths"] - s["offsets"].diff()).long()
    q = torch.zeros((B, m, case["heads"], d), device="cuda")
    q[seq, i] = s["q"][:n].float()
    # what a row sees: the context, and of the drafted tokens those that its mask names
    token = torch.arange(k.shape[1], device="cuda")[None, :]
    draft = token - ctx[seq][:, None]
    if case["chain"]:
        sees = draft <= i[:, None]
    else:
        bit = draft.clamp(0, 64 * s["masks"].shape[1] - 1)
        named = (torch.gather(s["masks"], 1, bit >> 6) >> (bit & 63)) & 1
        sees = (draft < 0) | ((named == 1) & (draft < s["offsets"].diff().long()[seq][:, None]))
    live = torch.zeros((B, m, k.shape[1]), device="cuda", dtype=torch.bool)
    live[seq, i] = sees
    scores = torch.matmul(q.view(B, m, hk, G, d).permute(0, 2, 1, 3, 4).flatten(2, 3), k.permute(0, 2, 3, 1))
    scores = scores.view(B, hk, m, G, -1).mul_(s["scale"])
    scores = scores.masked_fill_(~live[:, None, :, None, :], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(torch.isinf(top), 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3)).view(B, hk, m, G, d)
    o = (o / torch.where(total == 0, 1.0, total)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s["out"][:n] = o[seq, i].to(s["q"].dtype)
    if not case["lse"]:
        return s["out"]
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).flatten(2, 3)
    s["lse"][:n] = lse[seq, i]
    return s["out"], s["lse"]


def _plain_keep(s):
    ps = s["case"]["page_size"]
    path = s["path"].long()
    ctx = (s["lengths"] - s["offsets"].diff()).long()
    seq, k = (path >= 0).nonzero(as_tuple=True)
    src, dst = ctx[seq] + path[seq, k], ctx[seq] + k
    tables = s["tables"].long()
    s["pools"][:, :, tables[seq, dst // ps], dst % ps] = s["pools"][:, :, tables[seq, src // ps], src % ps]
    s["new_lengths"].copy_(ctx + (path >= 0).sum(1))
    return s["pools"], s["new_lengths"]


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"q4": _plain_q4, "tree": _plain_tree, "keep": _plain_keep}[op](state)
    import adapter_sgmv_lora_gb300 as lk
    if op == "q4":
        lk.lora_base_q4_apply(state["problem"], state["workspace"])
        return state["y"]
    if op == "tree":
        lk.lora_tree_attention(state["problem"], state["workspace"])
        return state["out"] if state["lse"] is None else (state["out"], state["lse"])
    lk.lora_kv_keep_rows(state["problem"])
    return state["pools"], state["new_lengths"]


# ------------------------------------------------------- 64-bit definition --

def _exact_q4(case, seed):
    s = _q4_data(case, seed)
    y = torch.zeros((s["T"], sum(s["outs"])), device="cuda", dtype=torch.float64)
    x = s["x"].double()
    for g in range(s["scales"].shape[1]):                         # group by group of the inputs
        lo, hi = g * case["group"], min((g + 1) * case["group"], case["in_dim"])
        j = torch.arange(lo, hi, device="cuda")
        code = (s["q"][:, j // 2] >> (4 * (j % 2)).to(torch.uint8)) & 15
        zero = s["zeros"][:, g:g + 1].double() if case["zeros"] else 8.0
        y += (x[:, lo:hi] @ (code.double() - zero).T) * s["scales"][:, g].double()
    for slot, lo, hi in zip(s["ids"], s["offs"][:-1], s["offs"][1:]):
        u = x[lo:hi] @ s["a"][slot].double().T
        col = 0
        for j, o in enumerate(s["outs"]):
            part = u[:, j * case["rank"]:(j + 1) * case["rank"]]
            y[lo:hi, col:col + o] += part @ s["b"][slot, col:col + o].double().T
            col += o
    return y


def _exact_tree(case, seed):
    s = _tree_data(case, seed)
    G = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.zeros(s["q"].shape[:2], device="cuda", dtype=torch.float64)
    at = 0
    for b, (n, c) in enumerate(zip(s["rows"], s["ctx"])):
        pages = s["tables"][b, :-(-(n + c) // case["page_size"])].long()
        k = s["kc"][pages].reshape(-1, case["kv_heads"], case["head_dim"])[:n + c].double()
        v = s["vc"][pages].reshape(-1, case["kv_heads"], case["head_dim"])[:n + c].double()
        hidden = torch.zeros((n, n + c), dtype=torch.bool, device="cuda")
        if case["chain"]:
            hidden[:, c:] = torch.ones((n, n), device="cuda").triu(1) > 0
        else:
            words = s["masks"][at:at + n].cpu().numpy().view(np.uint64)
            bits = np.unpackbits(words.view(np.uint8).reshape(n, -1), axis=1, bitorder="little")[:, :n]
            hidden[:, c:] = torch.from_numpy(bits == 0).cuda()
        for h in range(case["heads"]):
            z = s["q"][at:at + n, h].double() @ k[:, h // G].T / math.sqrt(case["head_dim"])
            z[hidden] = float("-inf")
            lse[at:at + n, h] = torch.logsumexp(z, -1)
            out[at:at + n, h] = torch.softmax(z, -1).nan_to_num(0.0) @ v[:, h // G]  # an empty row: zeros
        at += n
    return (out, lse) if case["lse"] else out


def exact(case, seed):
    if case["op"] == "q4":
        return _exact_q4(case, seed)
    if case["op"] == "tree":
        return _exact_tree(case, seed)
    return None  # moved rows compute no numbers


def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "q4":
        ids, offs, T = _routes(case)
        n, O, R = case["in_dim"], sum(_outs(case)), case["rank"]
        nR = len(_outs(case)) * R
        groups = -(-n // case["group"])
        nbytes = O * -(-n // 2) + O * groups * (es + (1 if case["zeros"] else 0)) + T * (n + O) * es
        nbytes += len(ids) * (nR * n + O * R) * es
        return {"bytes": nbytes, "flops": 2 * T * O * n + 2 * offs[-1] * (nR * n + O * R)}
    rows, ctx, _, _ = _shapes(case)
    hk, d = case["kv_heads"], case["head_dim"]
    if case["op"] == "tree":
        h = case["heads"]
        tokens = sum(rows) + sum(ctx)
        nbytes = 2 * tokens * hk * d * es + 2 * sum(rows) * h * d * es
        nbytes += 4 * sum(-(-(a + b) // case["page_size"]) for a, b in zip(rows, ctx)) + 8 * case["seqs"]
        nbytes += (0 if case["chain"] else 8 * sum(rows) * -(-max(rows) // 64)) + (4 * sum(rows) * h if case["lse"] else 0)
        return {"bytes": nbytes, "flops": 4 * h * d * sum(n * (c + n / 2) for n, c in zip(rows, ctx))}
    # half of the kept rows on average, read and written in every layer, an index each
    moved = sum(min(n, case["kept"]) for n in rows) // 2
    return {"bytes": 4 * moved * hk * d * es * case["layers"] + 4 * case["seqs"] * (case["kept"] + 4), "flops": 0}
