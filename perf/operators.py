"""The attention-side operators of the serving path, and their plain forms.

Between the fused q/k/v projection and o_proj a served layer rotates (and for
some models normalises) q and k, keeps k and v in a paged cache, attends to
the cache with one new token per sequence, and copies pages when sequences
fork or the cache is compacted.  Three operators do that:

  rope   lora_rope_append: per-head RMS norm of q and k, position rotation,
         q written out, k and v written into the cache's pages
  attn   lora_paged_attention: one new token per sequence over its pages
  pages  lora_kv_copy_pages: listed pages copied in every layer's K and V

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

def _rope(name, kind, tokens, heads, kv_heads, head_dim, rotary_dim, dtype="bf16", interleaved=False, norm=False,
          scaling="none", theta=500000.0, factor=8.0, attention_scale=1.0, max_position=8192, page_size=16,
          order="token", pad=0):
    return dict(name=name, op="rope", kind=kind, tokens=tokens, heads=heads, kv_heads=kv_heads, head_dim=head_dim,
                rotary_dim=rotary_dim, dtype=dtype, interleaved=interleaved, norm=norm, scaling=scaling, theta=theta,
                factor=factor, attention_scale=attention_scale, max_position=max_position, page_size=page_size,
                order=order, pad=pad)


def _attn(name, seqs, min_len, max_len, heads, kv_heads, head_dim, dtype="bf16", page_size=16, order="token",
          empty=0, lse=False, lengths_seed=1):
    return dict(name=name, op="attn", seqs=seqs, min_len=min_len, max_len=max_len, heads=heads, kv_heads=kv_heads,
                head_dim=head_dim, dtype=dtype, page_size=page_size, order=order, empty=empty, lse=lse,
                lengths_seed=lengths_seed)


def _pages(name, layers, num_pages, copies, kv_heads, head_dim, dtype="bf16", page_size=16, order="token",
           fork=False):
    return dict(name=name, op="pages", layers=layers, num_pages=num_pages, copies=copies, kv_heads=kv_heads,
                head_dim=head_dim, dtype=dtype, page_size=page_size, order=order, fork=fork)


def listed():
    return [
        # one token of one request: latency alone (8B attention: 32 query heads, 8 key/value heads, 128 wide)
        _rope("rope_1", "decode", 1, 32, 8, 128, 128),
        # a decode batch of 256 one-token requests at positions of a long context, with q/k norms; the last 13
        # rows only fill the batch up and go to no page
        _rope("rope_decode256_norm", "decode", 256, 32, 8, 128, 128, norm=True, scaling="linear", factor=4.0,
              max_position=131072, pad=13),
        # 8192 prompt tokens of the 70B attention (64 and 8 heads), frequencies scaled by parts
        _rope("rope_prefill70b", "prefill", 8192, 64, 8, 128, 128, scaling="parts", max_position=131072),
        # fp32, interleaved pairs over a part of an 80-wide head, odd token count, head-major pages
        _rope("rope_f32_partial", "prefill", 1777, 16, 16, 80, 32, dtype="f32", interleaved=True, theta=10000.0,
              scaling="ntk", attention_scale=1.1, page_size=24, order="head"),
        # one request with a short context: latency alone
        _attn("attn_1x517", 1, 517, 517, 32, 8, 128),
        # a decode batch of 256 ragged contexts on the 8B attention
        _attn("attn_256_8b", 256, 128, 2048, 32, 8, 128),
        # one request with a long context: the split over its length alone fills the GPU
        _attn("attn_1x131071", 1, 131071, 131071, 32, 8, 128, page_size=32, lse=True),
        # few long contexts on the 70B attention (8 query heads share a key/value head), head-major pages
        _attn("attn_24_70b", 24, 8192, 32768, 64, 8, 128, page_size=64, order="head"),
        # fp32 without shared heads, odd lengths, some batch entries empty
        _attn("attn_f32_ragged", 37, 1, 3001, 8, 8, 64, dtype="f32", page_size=8, empty=3),
        # copy on write of one forked request's last page, all layers of an 8B model
        _pages("pages_fork1", 32, 256, 1, 8, 128),
        # one prompt's last pages given to many forks (the same source many times)
        _pages("pages_fork_many", 32, 512, 192, 8, 128, fork=True),
        # a compaction of the cache: a thousand pages moved, all layers
        _pages("pages_compact", 32, 2048, 900, 8, 128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "pages"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    group = rng.choice([1, 3, 4, 4, 7, 8, 8, 16])
    heads = kv_heads * min(group, max(1, 64 // kv_heads))
    head_dim = rng.choice([32, 64, 80, 96, 128, 128, 128, 256])
    page_size = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    order = rng.choice(["token", "head"])
    if op == "rope":
        most = 8192 * 80 * 128 * 2 // ((heads + 2 * kv_heads) * head_dim * BYTES[dtype])
        tokens = _log_int(rng, 1, min(16384, max(1, most)))
        kind = "decode" if tokens <= 512 and rng.random() < 0.7 else "prefill"
        part = rng.choice([1, 1, 1, 2, 4])
        c = _rope(None, kind, tokens, heads, kv_heads, head_dim, head_dim // part, dtype=dtype,
                  interleaved=rng.random() < 0.4, norm=rng.random() < 0.5,
                  scaling=rng.choice(["none", "linear", "ntk", "parts"]),
                  theta=rng.choice([10000.0, 500000.0, 1000000.0]), factor=rng.choice([2.0, 4.0, 8.0, 32.0]),
                  attention_scale=rng.choice([1.0, 1.0, 1.2079]), max_position=_log_int(rng, 16, 1000000),
                  page_size=page_size, order=order, pad=rng.choice([0, 0, 1]) if tokens > 1 else 0)
    elif op == "attn":
        budget = 24 * 20000 * 8 * 128 * 2          # cache elements of the largest listed case, K and V each
        most = budget // 2 // (kv_heads * head_dim * BYTES[dtype])
        seqs = _log_int(rng, 1, 300)
        max_len = _log_int(rng, 1, max(1, min(131072, most // seqs)))
        min_len = max(1, max_len // rng.choice([1, 2, 16, 1000]))
        empty = rng.choice([0, 0, 1, 2]) if seqs > 3 else 0
        c = _attn(None, seqs, min_len, max_len, heads, kv_heads, head_dim, dtype=dtype, page_size=page_size,
                  order=order, empty=empty, lse=empty == 0 and rng.random() < 0.5,
                  lengths_seed=rng.randrange(1 << 30))
    else:
        page_bytes = page_size * kv_heads * head_dim * BYTES[dtype]
        layers = _log_int(rng, 1, 80)
        most = int(32 * 900 * 16 * 8 * 128 * 2 // (page_bytes * layers))
        copies = _log_int(rng, 1, max(1, min(4000, most)))
        c = _pages(None, layers, 2 * copies + rng.randrange(1, 40), copies, kv_heads, head_dim, dtype=dtype,
                   page_size=page_size, order=order, fork=rng.random() < 0.4)
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


def _pool(case, num_pages, g, fill=True):
    """One layer's K or V pages as a [pages, page_size, kv_heads, head_dim] view of token-major or head-major
    memory."""
    ps, h, d, dt = case["page_size"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    shape = (num_pages, ps, h, d) if case["order"] == "token" else (num_pages, h, ps, d)
    t = _randn(shape, g, dt) if fill else torch.zeros(shape, device="cuda", dtype=dt)
    return t if case["order"] == "token" else t.permute(0, 2, 1, 3)


def _lengths(case):
    r = random.Random(case["lengths_seed"])
    n = case["seqs"] - case["empty"]
    return [r.randint(case["min_len"], case["max_len"]) for _ in range(n)] + [0] * case["empty"]


def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    D, theta = case["rotary_dim"], case["theta"]
    i = np.arange(D // 2, dtype=np.float64)
    if case["scaling"] == "ntk":
        theta = theta * case["factor"] ** (D / (D - 2))
    f = theta ** (-2.0 * i / D)
    if case["scaling"] == "linear":
        f = f / case["factor"]
    elif case["scaling"] == "parts":
        # pairs that turn often within the original 8192 positions keep their frequency, slow ones are divided
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = keep * f + (1 - keep) * f / case["factor"]
    return f


def _rope_data(case, seed):
    g = _gen(seed)
    r = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    T, h, hk, d, ps = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], case["page_size"]
    # the rows the fused projection leaves: q | k | v
    qkv = _randn((T, (h + 2 * hk) * d), g, dt)
    q = qkv[:, :h * d].view(T, h, d)
    k = qkv[:, h * d:(h + hk) * d].view(T, hk, d)
    v = qkv[:, (h + hk) * d:].view(T, hk, d)
    used = -(-T // ps) + 1
    num_pages = used + 5
    order = np.array(r.sample(range(num_pages), used), dtype=np.int64)
    slot = np.arange(T)
    if case["kind"] == "decode":
        positions = np.array([r.randrange(case["max_position"]) for _ in range(T)], dtype=np.int64)
        slot = np.array(r.sample(range(used * ps), T), dtype=np.int64)
    else:
        # a few prompts, each from some position on
        positions = np.zeros(T, dtype=np.int64)
        cuts = sorted({0, T} | {r.randrange(T) for _ in range(min(T, 5))})
        for a, b in zip(cuts[:-1], cuts[1:]):
            positions[a:b] = r.randrange(max(1, case["max_position"] - (b - a))) + np.arange(b - a)
    rows = order[slot // ps] * ps + slot % ps
    if case["pad"]:
        rows[T - case["pad"]:] = -1
    w = [1.0 + 0.2 * _randn((d,), g, torch.float32) for _ in range(2)]
    w = [t.to(dt) for t in w] if case["norm"] else [None, None]
    return dict(q=q, k=k, v=v, positions=torch.from_numpy(positions.astype(np.int32)).cuda(),
                rows=torch.from_numpy(rows.astype(np.int32)).cuda(), qw=w[0], kw=w[1], num_pages=num_pages, eps=1e-6)


def _attn_data(case, seed):
    g = _gen(seed)
    r = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    ps = case["page_size"]
    lens = _lengths(case)
    r.shuffle(lens)
    need = [-(-n // ps) for n in lens]
    num_pages = sum(need) + 3
    ids = list(range(num_pages))
    r.shuffle(ids)
    max_pages = max(1, max(need))
    tables = np.full((case["seqs"], max_pages), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
    q = _randn((case["seqs"], case["heads"], case["head_dim"]), g, dt, 1.5)
    kc = _pool(case, num_pages, g)
    vc = _pool(case, num_pages, g)
    return dict(q=q, kc=kc, vc=vc, lens=lens, tables=torch.from_numpy(tables).cuda(),
                lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def _pages_data(case, seed):
    g = _gen(seed)
    r = random.Random(seed)
    n = case["copies"]
    ids = r.sample(range(case["num_pages"]), min(2 * n, case["num_pages"]))
    if case["fork"]:
        # a few source pages, each to many destinations
        few = max(1, n // 16)
        src = [ids[i % few] for i in range(n)]
        dst = ids[few:few + n]
    else:
        src, dst = ids[:n], ids[n:2 * n]
    pools = [(_pool(case, case["num_pages"], g), _pool(case, case["num_pages"], g)) for _ in range(case["layers"])]
    return dict(pools=pools, src=np.array(src, dtype=np.int32), dst=np.array(dst, dtype=np.int32))


def prepare(case, seed):
    if case["op"] == "rope":
        s = _rope_data(case, seed)
        g = _gen(seed + 1)
        s["kc"] = _pool(case, s["num_pages"], g)
        s["vc"] = _pool(case, s["num_pages"], g)
        s["q_out"] = torch.empty(s["q"].shape, device="cuda", dtype=s["q"].dtype)
        if own:
            import adapter_sgmv_lora_gb300 as lk
            rope = lk.lora_build_rope(case["rotary_dim"], case["theta"], scaling=case["scaling"],
                                      factor=case["factor"], original_max_positions=8192, low_turns=1.0,
                                      high_turns=4.0, attention_scale=case["attention_scale"])
            s["problem"] = lk.RopeProblem(q=s["q"], k=s["k"], v=s["v"], q_out=s["q_out"],
                                          rope=lk.rope_to_device(rope), positions=s["positions"],
                                          interleaved=case["interleaved"], cache=lk.KVCache(s["kc"], s["vc"]),
                                          cache_rows=s["rows"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"])
        else:
            turns = np.array([int(f / (2 * math.pi) * 2.0 ** 64) for f in _frequencies(case)], dtype=np.uint64)
            s["turns"] = torch.from_numpy(turns.view(np.int64)).cuda()
    elif case["op"] == "attn":
        s = _attn_data(case, seed)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda") if case["lse"] else None
        s["scale"] = 1.0 / math.sqrt(case["head_dim"])
        if own:
            import adapter_sgmv_lora_gb300 as lk
            s["problem"] = lk.AttentionProblem(q=s["q"], out=s["out"], cache=lk.KVCache(s["kc"], s["vc"]),
                                               block_tables=s["tables"], lengths=s["lengths"], scale=s["scale"],
                                               lse=s["lse"])
            s["workspace"] = lk.new_attention_workspace(s["problem"])
    else:
        s = _pages_data(case, seed)
        if own:
            import adapter_sgmv_lora_gb300 as lk
            s["caches"] = lk.KVCaches([lk.KVCache(k, v) for k, v in s["pools"]])
        else:
            s["src_ids"] = torch.from_numpy(s["src"]).cuda().long()
            s["dst_ids"] = torch.from_numpy(s["dst"]).cuda().long()
    s["case"] = case
    return s


# ------------------------------------------------------------ plain forms --

def _plain_rotate(x, w, cos, sin, case, eps):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    D = case["rotary_dim"]
    a = x[..., 0:D:2] if case["interleaved"] else x[..., :D // 2]
    b = x[..., 1:D:2] if case["interleaved"] else x[..., D // 2:D]
    ra, rb = a * cos - b * sin, a * sin + b * cos
    rot = torch.stack((ra, rb), -1).flatten(-2) if case["interleaved"] else torch.cat((ra, rb), -1)
    return torch.cat((rot, x[..., D:]), -1)


def _plain_rope(s):
    case = s["case"]
    dt = s["q"].dtype
    # turns are fractions of 2^64: the wrapped integer product is the exact fractional turn
    phase = (s["positions"].long()[:, None] * s["turns"][None, :]) >> 32
    angle = phase.float() * (math.pi / 2.0 ** 31)
    cos = (torch.cos(angle) * case["attention_scale"])[:, None, :]
    sin = (torch.sin(angle) * case["attention_scale"])[:, None, :]
    s["q_out"].copy_(_plain_rotate(s["q"], s["qw"], cos, sin, case, s["eps"]))
    k = _plain_rotate(s["k"], s["kw"], cos, sin, case, s["eps"])
    n = case["tokens"] - case["pad"]
    rows = s["rows"][:n].long()
    page, off = rows // case["page_size"], rows % case["page_size"]
    s["kc"][page, off] = k[:n].to(dt)
    s["vc"][page, off] = s["v"][:n]
    return s["q_out"], s["kc"], s["vc"]


def _plain_attn(s):
    case = s["case"]
    B, hk = case["seqs"], case["kv_heads"]
    G, d = case["heads"] // hk, case["head_dim"]
    tables = s["tables"].clamp(min=0).long()
    k = s["kc"][tables].flatten(1, 2).float()                     # [B, L, hk, d]
    v = s["vc"][tables].flatten(1, 2).float()
    live = torch.arange(k.shape[1], device="cuda")[None, :] < s["lengths"][:, None]
    q = s["q"].float().view(B, hk, G, d)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]  # [B, hk, G, L]
    scores = torch.where(live[:, None, None, :], scores, float("-inf"))
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(m), 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(l == 0, 1.0, l)
    s["out"].copy_(o.reshape(B, case["heads"], d))
    if not case["lse"]:
        return s["out"]
    s["lse"].copy_((m + torch.log(l)).reshape(B, case["heads"]))
    return s["out"], s["lse"]


def _plain_pages(s):
    for k, v in s["pools"]:
        k[s["dst_ids"]] = k[s["src_ids"]]
        v[s["dst_ids"]] = v[s["src_ids"]]
    return [t for kv in s["pools"] for t in kv]


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "attn": _plain_attn, "pages": _plain_pages}[op](state)
    import adapter_sgmv_lora_gb300 as lk
    if op == "rope":
        lk.lora_rope_append(state["problem"])
        return state["q_out"], state["kc"], state["vc"]
    if op == "attn":
        lk.lora_paged_attention(state["problem"], state["workspace"])
        return state["out"] if state["lse"] is None else (state["out"], state["lse"])
    lk.lora_kv_copy_pages(state["caches"], state["src"], state["dst"])
    return [t for kv in state["pools"] for t in kv]


# ------------------------------------------------------- 64-bit definition --

def _exact_rope(case, seed):
    s = _rope_data(case, seed)
    g = _gen(seed + 1)
    kc, vc = _pool(case, s["num_pages"], g).double(), _pool(case, s["num_pages"], g).double()
    f = torch.from_numpy(_frequencies(case)).cuda()
    D, m = case["rotary_dim"], case["attention_scale"]
    angle = s["positions"].double()[:, None] * f[None, :]
    c, sn = torch.cos(angle)[:, None] * m, torch.sin(angle)[:, None] * m

    def turn(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(torch.mean(y * y, -1, keepdim=True) + s["eps"]) * w.double()
        o = y.clone()
        first = slice(0, D, 2) if case["interleaved"] else slice(0, D // 2)
        second = slice(1, D, 2) if case["interleaved"] else slice(D // 2, D)
        o[..., first] = c * y[..., first] - sn * y[..., second]
        o[..., second] = sn * y[..., first] + c * y[..., second]
        return o

    k = turn(s["k"], s["kw"])
    keep = s["rows"] >= 0
    rows = s["rows"][keep].long()
    at = (torch.div(rows, case["page_size"], rounding_mode="floor"), rows % case["page_size"])
    kc[at] = k[keep]
    vc[at] = s["v"][keep].double()
    return turn(s["q"], s["qw"]), kc, vc


def _exact_attn(case, seed):
    s = _attn_data(case, seed)
    G = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full(s["q"].shape[:2], float("-inf"), device="cuda", dtype=torch.float64)
    for b, n in enumerate(s["lens"]):
        if n == 0:
            continue
        pages = s["tables"][b, :-(-n // case["page_size"])].long()
        k = s["kc"][pages].reshape(-1, case["kv_heads"], case["head_dim"])[:n].double()
        v = s["vc"][pages].reshape(-1, case["kv_heads"], case["head_dim"])[:n].double()
        for j in range(case["kv_heads"]):
            z = s["q"][b, j * G:(j + 1) * G].double() @ k[:, j].T / math.sqrt(case["head_dim"])
            lse[b, j * G:(j + 1) * G] = torch.logsumexp(z, -1)
            out[b, j * G:(j + 1) * G] = torch.softmax(z, -1) @ v[:, j]
    return (out, lse) if case["lse"] else out


def exact(case, seed):
    if case["op"] == "rope":
        return _exact_rope(case, seed)
    if case["op"] == "attn":
        return _exact_attn(case, seed)
    return None  # a copy computes no numbers


def work(case):
    es = BYTES[case["dtype"]]
    h, hk, d = case.get("heads", 0), case["kv_heads"], case["head_dim"]
    if case["op"] == "rope":
        # q, k, v read and written once, a position and a row per token; norm 3 and rotation 3 per element
        T = case["tokens"]
        stored = T - case["pad"]
        nbytes = T * (h + 2 * hk) * d * es + T * h * d * es + 2 * stored * hk * d * es + 8 * T
        flops = T * (h + hk) * (3 * case["rotary_dim"] + (3 * d if case["norm"] else 0))
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "attn":
        lens = _lengths(case)
        n = sum(lens)
        pages = sum(-(-x // case["page_size"]) for x in lens)
        nbytes = 2 * n * hk * d * es + 2 * case["seqs"] * h * d * es + 4 * pages + 4 * case["seqs"]
        nbytes += 4 * case["seqs"] * h if case["lse"] else 0
        return {"bytes": nbytes, "flops": 4 * n * h * d}
    page = case["page_size"] * hk * d * es
    sources = max(1, case["copies"] // 16) if case["fork"] else case["copies"]
    return {"bytes": 2 * case["layers"] * page * (sources + case["copies"]), "flops": 0}
