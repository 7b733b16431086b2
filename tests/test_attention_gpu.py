"""Rotation + cache append, paged attention and page copies on the GPU against
their definitions in 64 bits (numpy), at the sizes, layouts and masks where
they can go wrong.

Bounds, with e = 2^-24 (fp32's half ulp at 1) and h = 2^-8 (bf16's, relative):
  rotation   the angle is exact to 2^-31 half turns before its fp32 rounding,
             so sin and cos are off by a few e; a rotated element is two
             products and a sum: 16 e (|a| + |b|) s.  A norm adds the sum of
             head_dim squares (head_dim / 2 + 8) e.
  attention  a score is a sum of head_dim products: (head_dim + 8) e times
             scale sum |q k|, and a probability is off by as much relatively;
             the output is a sum of len products over a sum of len: (2 len +
             16) e.  Times the weighted mean of |v|.  The bf16 path's
             probabilities have 16 significant bits: 2^-16 more.
  rounding   bf16 results: h |ref| on top; both also 2^-126 (subnormals).
"""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: E}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as ge
    ge.build()


@pytest.fixture(autouse=True)
def _status_clean():
    yield
    assert lk.lora_get_device_status() == 0


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def pool(num_pages, ps, heads, hd, dtype, order, fill=float("nan")):
    """K and V views [pages, ps, heads, hd] of one of the memory layouts."""
    if order == "token":
        t = [torch.full((num_pages, ps, heads, hd), fill, dtype=dtype, device="cuda") for _ in range(2)]
    elif order == "head":
        t = [torch.full((num_pages, heads, ps, hd), fill, dtype=dtype, device="cuda").permute(0, 2, 1, 3)
             for _ in range(2)]
    elif order == "side":     # K and V side by side within a token
        both = torch.full((num_pages, ps, 2, heads, hd), fill, dtype=dtype, device="cuda")
        t = [both[:, :, 0], both[:, :, 1]]
    elif order == "gap":      # rows with a gap of 3 elements: nothing on a 16-byte boundary
        t = [torch.full((num_pages, ps, heads, hd + 3), fill, dtype=dtype, device="cuda")[..., :hd] for _ in range(2)]
    else:
        raise ValueError(order)
    return t


# --------------------------------------------------------------- rotation --

def rope_reference(x, w, positions, freqs, rot, interleaved, scale, eps):
    """(value, sum of magnitudes) in 64 bits; x [T, H, hd]."""
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * w
    out, mag = y.copy(), np.abs(y)
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    ang = positions.astype(np.float64)[:, None] * freqs[None, :]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    out[..., a] = scale * (y[..., a] * c - y[..., b] * s)
    out[..., b] = scale * (y[..., a] * s + y[..., b] * c)
    m = abs(scale) * (np.abs(y[..., a]) + np.abs(y[..., b]))
    mag[..., a] = m
    mag[..., b] = m
    return out, mag


ROPE_CASES = [
    # dtype, T, H, Hk, hd, rot, interleaved, norm, order, page_size, fused, attention scale
    (BF, 1, 32, 8, 128, 128, False, False, "token", 16, True, 1.0),
    (BF, 37, 8, 2, 128, 128, False, True, "head", 16, True, 1.0),
    (BF, 5, 4, 4, 128, 64, False, True, "token", 8, True, 1.25),
    (BF, 9, 4, 2, 64, 64, True, False, "side", 1, True, 1.0),
    (BF, 300, 6, 2, 80, 40, True, True, "token", 24, True, 1.1),
    (BF, 11, 3, 1, 80, 48, False, False, "head", 16, True, 1.0),
    (BF, 7, 2, 2, 256, 256, False, True, "token", 16, True, 1.0),
    (BF, 13, 5, 1, 96, 24, False, True, "token", 16, True, 1.0),   # 12 pairs: not a whole 16 bytes of a half
    (BF, 13, 5, 1, 33, 32, False, True, "token", 16, False, 1.0),  # odd width
    (BF, 6, 2, 1, 2, 2, True, False, "gap", 4, False, 1.0),
    (BF, 6, 16, 16, 64, 64, False, False, "gap", 4, True, 1.0),    # unaligned cache rows
    (F32, 1, 8, 8, 16, 16, False, False, "token", 16, True, 1.0),
    (F32, 101, 8, 4, 128, 128, False, True, "head", 16, True, 1.0),
    (F32, 29, 16, 16, 80, 32, True, False, "side", 24, True, 1.1),
    (F32, 10, 3, 3, 256, 256, True, True, "token", 5, True, 1.0),
    (F32, 10, 3, 3, 20, 6, False, True, "token", 5, True, 1.0),
    (F32, 10, 3, 3, 7, 4, True, True, "gap", 5, False, 1.0),
]


def make_qkv(T, H, Hk, hd, dtype, seed, fused):
    if fused:
        y = randn((T, (H + 2 * Hk) * hd), dtype, seed)
        return (y[:, :H * hd].unflatten(1, (H, hd)), y[:, H * hd:(H + Hk) * hd].unflatten(1, (Hk, hd)),
                y[:, (H + Hk) * hd:].unflatten(1, (Hk, hd)))
    return tuple(randn((T, n, hd), dtype, seed + i) for i, n in enumerate((H, Hk, Hk)))


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "-".join(str(x) for x in c[:10]).replace("torch.", ""))
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_append(case, in_place):
    dtype, T, H, Hk, hd, rot, inter, norm, order, ps, fused, ascale = case
    q, k, v = make_qkv(T, H, Hk, hd, dtype, 3, fused)
    q0, k0, v0 = f64(q), f64(k), v.clone()
    rng = np.random.default_rng(5)
    positions = rng.integers(0, 200000, size=T)
    positions[0] = 0
    if T > 4:
        positions[1:5] = [1, 2 ** 31 - 1, -3, 1048576]
    freqs = 500000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    rope = lk.rope_to_device(lk.lora_build_rope(rot, 500000.0, attention_scale=ascale))
    num_pages = T // ps + 3
    rows = rng.permutation(num_pages * ps)[:T]
    if T > 6:
        rows[6] = -1
    kc, vc = pool(num_pages, ps, Hk, hd, dtype, order, fill=7.0)
    qw = randn((hd,), dtype, 8) if norm else None
    kw = randn((hd,), dtype, 9) if norm else None
    q_out = q if in_place else torch.full((T, H, hd), float("nan"), dtype=dtype, device="cuda")
    k_out = k if in_place else torch.full((T, Hk, hd), float("nan"), dtype=dtype, device="cuda")
    prob = lk.RopeProblem(q=q, k=k, v=v, q_out=q_out, k_out=k_out, rope=rope, interleaved=inter,
                          positions=torch.tensor(positions, dtype=torch.int32, device="cuda"),
                          cache=lk.KVCache(kc, vc),
                          cache_rows=torch.tensor(rows, dtype=torch.int32, device="cuda"), q_weight=qw, k_weight=kw)
    lk.lora_rope_append(prob)
    v_elems = 8 if dtype == BF else 4      # per 16 bytes
    fast = fused and order != "gap" and hd % v_elems == 0 and rot % (v_elems if inter else 2 * v_elems) == 0
    assert lk.lora_last_call_path() == (lk.PATH_ROPE if fast else lk.PATH_GENERIC_ROPE, 1)
    torch.cuda.synchronize()
    ascale = float(np.float32(ascale))
    eps = float(np.float32(1e-6))
    tol = (16 + (hd / 2 + 8 if norm else 0)) * E
    for got, x, w, n in ((q_out, q0, qw, "q"), (k_out, k0, kw, "k")):
        ref, mag = rope_reference(x, None if w is None else f64(w), positions, freqs, rot, inter, ascale, eps)
        err = np.abs(f64(got) - ref)
        assert np.all(err <= tol * mag + ROUND[dtype] * np.abs(ref) * (1 + 1e-3) + 2.0 ** -126), (n, err.max())
    # the cache: exactly k_out and v at the rows, everything else untouched
    want_k, want_v = pool(num_pages, ps, Hk, hd, dtype, order, fill=7.0)
    for t in range(T):
        if rows[t] >= 0:
            want_k[rows[t] // ps, rows[t] % ps] = k_out[t]
            want_v[rows[t] // ps, rows[t] % ps] = v0[t]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_rope_parts_of_the_call():
    """q alone, k alone, no rotation, no tokens; the fast and the generic kernel agree on the same numbers."""
    T, H, Hk, hd = 19, 4, 2, 64
    q, k, v = make_qkv(T, H, Hk, hd, BF, 1, True)
    rope = lk.rope_to_device(lk.lora_build_rope(hd))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    full_q, full_k = torch.empty_like(q), torch.empty_like(k)
    lk.lora_rope_append(lk.RopeProblem(q=q, k=k, q_out=full_q, k_out=full_k, rope=rope, positions=pos))
    only_q, only_k = torch.empty_like(q), torch.empty_like(k)
    lk.lora_rope_append(lk.RopeProblem(q=q, q_out=only_q, rope=rope, positions=pos))
    lk.lora_rope_append(lk.RopeProblem(k=k, k_out=only_k, rope=rope, positions=pos))
    assert torch.equal(full_q, only_q) and torch.equal(full_k, only_k)
    # rows two elements apart in memory from a 16-byte boundary
    wide = torch.zeros((T, H, hd + 2), dtype=BF, device="cuda")
    wide[..., 2:] = q
    odd = torch.empty_like(wide)[..., 2:]
    lk.lora_rope_append(lk.RopeProblem(q=wide[..., 2:], q_out=odd, rope=rope, positions=pos))
    assert lk.lora_last_call_path()[0] == lk.PATH_GENERIC_ROPE
    assert (odd.float() - full_q.float()).abs().max() <= 2.0 ** -8 * full_q.float().abs().max()
    plain = torch.empty_like(q)
    lk.lora_rope_append(lk.RopeProblem(q=q, q_out=plain))
    assert torch.equal(plain, q)
    empty = torch.empty((0, H, hd), dtype=BF, device="cuda")
    lk.lora_rope_append(lk.RopeProblem(q=empty, q_out=empty, rope=rope, positions=pos[:0]))
    assert lk.lora_last_call_path() == (0, 0)


def test_rope_broadcast_key():
    """One key row shared by all heads through a stride of 0."""
    T, Hk, hd = 12, 4, 128
    one = randn((T, 1, hd), BF, 2)
    rope = lk.rope_to_device(lk.lora_build_rope(hd))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    a, b = (torch.empty((T, Hk, hd), dtype=BF, device="cuda") for _ in range(2))
    lk.lora_rope_append(lk.RopeProblem(k=one.expand(T, Hk, hd), k_out=a, rope=rope, positions=pos))
    lk.lora_rope_append(lk.RopeProblem(k=one.expand(T, Hk, hd).contiguous(), k_out=b, rope=rope, positions=pos))
    assert torch.equal(a, b)


def test_rope_bad_cache_rows():
    T, H, hd, ps = 6, 2, 64, 4
    q, k, v = make_qkv(T, H, H, hd, BF, 1, True)
    kc, vc = pool(3, ps, H, hd, BF, "token", fill=1.0)
    rows = torch.tensor([0, 12, -2, 2 ** 31 - 1, 11, -2 ** 31], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    lk.lora_rope_append(lk.RopeProblem(q=q, k=k, v=v, q_out=out, cache=lk.KVCache(kc, vc), cache_rows=rows))
    assert lk.lora_get_device_status() == lk.DEV_BAD_PAGE
    assert torch.equal(out, q)
    want = torch.ones_like(vc)
    want[0, 0], want[2, 3] = v[0], v[4]
    assert torch.equal(vc, want)


# -------------------------------------------------------------- attention --

def attention_reference(q, k, v, scale):
    """(out, lse, bound) in 64 bits of one sequence: q [H, hd], k and v [n, Hk, hd]."""
    H, hd = q.shape
    n, Hk, _ = k.shape
    out, lse, bound = np.zeros((H, hd)), np.full(H, -np.inf), np.zeros((H, hd))
    for h in range(H):
        if n == 0:
            continue
        kk, vv = k[:, h // (H // Hk)], v[:, h // (H // Hk)]
        s = scale * (kk @ q[h])
        m = s.max()
        p = np.exp(s - m)
        out[h] = p @ vv / p.sum()
        lse[h] = m + np.log(p.sum())
        ds = (hd + 8) * E * (abs(scale) * (np.abs(kk) @ np.abs(q[h]))).max()
        bound[h] = (2 * ds + (2 * n + 16) * E) * (p @ np.abs(vv) / p.sum())
    return out, lse, bound


def make_attention(lens, H, Hk, hd, ps, dtype, order, seed=0, spare=2, scale_q=1.5, max_pages=None):
    """Paged K/V with NaN wherever no sequence has a token, tables with nonsense past each sequence's pages."""
    rng = np.random.default_rng(seed)
    need = [-(-n // ps) for n in lens]
    num_pages = sum(need) + spare
    ids = rng.permutation(num_pages)
    M = max([1] + need) if max_pages is None else max_pages
    tables = rng.integers(-2 ** 31, 2 ** 31 - 1, size=(len(lens), M))
    kc, vc = pool(num_pages, ps, Hk, hd, dtype, order)
    ks, vs, at = [], [], 0
    for b, n in enumerate(lens):
        mine = ids[at:at + need[b]]
        at += need[b]
        tables[b, :need[b]] = mine
        kk, vv = randn((n, Hk, hd), dtype, seed * 1000 + 2 * b), randn((n, Hk, hd), dtype, seed * 1000 + 2 * b + 1)
        if n:
            pg = torch.from_numpy(mine[np.arange(n) // ps]).cuda()
            off = torch.arange(n, device="cuda") % ps
            kc[pg, off] = kk
            vc[pg, off] = vv
        ks.append(kk)
        vs.append(vv)
    q = randn((len(lens), H, hd), dtype, seed + 77, scale_q)
    return dict(q=q, k=ks, v=vs, cache=lk.KVCache(kc, vc), lens=lens,
                tables=torch.tensor(tables, dtype=torch.int32, device="cuda"),
                lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"))


def run_attention(a, q=None, out=None, with_lse=True, scale=None, stream=None):
    q = a["q"] if q is None else q
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], float("nan"), device="cuda") if with_lse else None
    prob = lk.AttentionProblem(q=q, out=out, cache=a["cache"], block_tables=a["tables"], lengths=a["lengths"],
                               scale=scale, lse=lse)
    ws = lk.new_attention_workspace(prob)
    ws.fill_(float("nan"))
    if stream is None:
        lk.lora_paged_attention(prob, ws)
    else:
        stream.wait_stream(torch.cuda.current_stream())
        lk.lora_paged_attention(prob, ws, stream=stream)
        torch.cuda.current_stream().wait_stream(stream)
    return out, lse


def check_attention(a, out, lse, scale, rows=None):
    dtype = a["q"].dtype
    for b in range(len(a["lens"])) if rows is None else rows:
        ref, rl, bound = attention_reference(f64(a["q"][b]), f64(a["k"][b]), f64(a["v"][b]), scale)
        got = f64(out[b])
        if dtype == BF:
            mean_v = bound * 0
            if a["lens"][b]:
                mean_v = np.abs(f64(a["v"][b])).max()
            bound = bound + 2.0 ** -16 * mean_v
        err = np.abs(got - ref)
        assert np.all(err <= bound + ROUND[dtype] * np.abs(ref) * (1 + 1e-3) + 2.0 ** -126), (b, a["lens"][b], err.max())
        if lse is None:
            continue
        if a["lens"][b] == 0:
            assert np.all(np.isneginf(f64(lse[b]))) and np.all(got == 0)
        else:
            hd = a["q"].shape[2]
            k64, q64 = np.abs(f64(a["k"][b])), np.abs(f64(a["q"][b]))
            most = scale * max((k64[:, h // (q64.shape[0] // k64.shape[1])] @ q64[h]).max()
                               for h in range(q64.shape[0]))
            tol = ((hd + 8) * most + 2 * a["lens"][b] + 16 + 4 * np.abs(rl)) * E
            assert np.all(np.abs(f64(lse[b]) - rl) <= tol), (b, np.abs(f64(lse[b]) - rl).max())


RAGGED = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 130, 257, 1000, 0]
ATTENTION_CASES = [
    # dtype, lens, H, Hk, hd, page_size, order
    (BF, RAGGED, 32, 8, 128, 16, "token"),
    (BF, RAGGED, 8, 1, 128, 16, "head"),
    (BF, RAGGED, 4, 4, 64, 1, "token"),
    (BF, RAGGED, 14, 2, 64, 24, "side"),      # 7 query heads a group
    (BF, RAGGED, 18, 2, 128, 3, "token"),     # 9 a group
    (BF, RAGGED, 32, 2, 128, 64, "token"),    # 16 a group
    (BF, RAGGED, 20, 1, 96, 16, "head"),      # 20 a group
    (BF, RAGGED, 71, 1, 64, 16, "token"),     # 71 a group
    (BF, RAGGED, 6, 2, 80, 8, "token"),
    (BF, RAGGED, 8, 2, 256, 16, "token"),
    (BF, RAGGED, 32, 2, 256, 16, "head"),
    (BF, RAGGED, 4, 2, 32, 16, "token"),
    (BF, RAGGED, 4, 2, 16, 16, "token"),
    (BF, RAGGED, 4, 2, 40, 16, "token"),
    (BF, RAGGED, 4, 2, 33, 16, "token"),      # odd width
    (BF, RAGGED, 4, 2, 64, 16, "gap"),        # rows off 16-byte boundaries
    (F32, RAGGED, 8, 8, 16, 16, "token"),
    (F32, RAGGED, 8, 2, 128, 16, "head"),
    (F32, RAGGED, 10, 1, 64, 5, "side"),
    (F32, RAGGED, 4, 4, 256, 16, "token"),
    (F32, RAGGED, 9, 3, 100, 16, "token"),
    (F32, RAGGED, 3, 3, 7, 2, "gap"),
    (BF, [1], 32, 8, 128, 16, "token"),
    (BF, [0], 32, 8, 128, 16, "token"),
    (BF, [0, 0, 0], 8, 8, 64, 16, "token"),
    (F32, [0], 8, 8, 64, 16, "token"),
    (BF, [3000], 32, 8, 128, 16, "token"),    # one context over many CTAs
    (BF, [20000], 4, 1, 128, 64, "token"),
    (F32, [5003], 4, 2, 128, 16, "token"),
    (BF, [9000, 1, 0, 5], 8, 2, 128, 16, "head"),
    (BF, [40] * 300, 8, 8, 64, 16, "token"),  # more streams than CTAs
    (BF, [1] * 700, 4, 4, 64, 16, "token"),
    (F32, [5] * 400, 4, 4, 64, 16, "token"),
]


@pytest.mark.parametrize("case", ATTENTION_CASES,
                         ids=lambda c: "%s-%dseq-%d-%d-%d-%d-%s" % (str(c[0])[6:], len(c[1]), *c[2:]))
def test_attention(case):
    dtype, lens, H, Hk, hd, ps, order = case
    a = make_attention(lens, H, Hk, hd, ps, dtype, order)
    out, lse = run_attention(a)
    mma = dtype == BF and hd % 8 == 0 and ps % 8 == 0 and order != "gap"
    core = lk.PATH_MMA_ATTENTION if mma else lk.PATH_GENERIC_ATTENTION
    assert lk.lora_last_call_path()[0] & ~lk.PATH_JOIN == core
    check_attention(a, out, lse, 1.0 / hd ** 0.5, rows=range(0, len(lens), max(1, len(lens) // 40)))


@pytest.mark.parametrize("dtype,lens,H,Hk,hd,ps,order", [
    (BF, [8 + 37 * i % 129 for i in range(145)] + [0], 64, 8, 128, 1, "token"),
    (BF, [8 + 37 * i % 129 for i in range(145)] + [0], 64, 8, 80, 1, "head"),
    (BF, [300 + 37 * i % 129 for i in range(60)], 32, 16, 128, 24, "token"),
    (BF, [5 + 53 * i % 400 for i in range(200)], 16, 8, 64, 3, "token"),
    (BF, [5 + 53 * i % 400 for i in range(100)], 32, 8, 32, 8, "side"),
    (BF, [5 + 53 * i % 200 for i in range(100)], 16, 8, 256, 5, "token"),
    (BF, [5 + 53 * i % 200 for i in range(100)], 64, 4, 128, 1, "token"),
    (F32, [5 + 53 * i % 200 for i in range(100)], 8, 8, 64, 3, "token"),
    (F32, [5 + 53 * i % 200 for i in range(100)], 32, 8, 128, 1, "token"),
    (BF, [1 + 11 * i % 128 for i in range(200)], 16, 4, 128, 1, "token"),   # warps on their own, up to 8 tiles
    (BF, [1 + 11 * i % 128 for i in range(200)], 16, 4, 128, 16, "token"),
    (BF, [900 + 53 * i % 400 for i in range(24)], 32, 8, 128, 16, "token"),
    (BF, [900 + 53 * i % 400 for i in range(24)], 64, 8, 128, 16, "head"),
    (BF, [8 + 37 * i % 129 for i in range(145)] + [0], 64, 8, 128, 8, "token"),
    (BF, [900 + 53 * i % 400 for i in range(24)], 16, 8, 64, 24, "token"),
    (BF, [300 + 53 * i % 200 for i in range(24)], 64, 4, 256, 8, "token"),
    (BF, [300 + 53 * i % 200 for i in range(30)], 18, 2, 128, 40, "head"),
    (BF, [900 + 53 * i % 400 for i in range(24)], 16, 8, 64, 32, "token"),
    (BF, [300 + 53 * i % 200 for i in range(24)], 64, 4, 256, 16, "token"),
    (BF, [300 + 53 * i % 200 for i in range(50)], 8, 8, 32, 16, "token"),
    (BF, [1 + 11 * i % 256 for i in range(200)], 8, 4, 64, 5, "head"),
    (F32, [1 + 11 * i % 64 for i in range(200)], 16, 4, 128, 3, "token"),
    (BF, [1 + 37 * i % 256 for i in range(300)], 32, 4, 128, 16, "token"),  # up to 16 tiles
    (BF, [1 + 37 * i % 256 for i in range(200)], 18, 2, 256, 8, "head"),
    (F32, [1 + 37 * i % 256 for i in range(300)], 4, 4, 128, 16, "token"),
])
def test_attention_many_streams_a_block(dtype, lens, H, Hk, hd, ps, order):
    """Several streams to every block, each of several tiles, with pages that end inside a tile: the lanes of a
    warp look different pages up on the way from one stream to the next."""
    a = make_attention(lens, H, Hk, hd, ps, dtype, order, seed=12)
    out, lse = run_attention(a)
    check_attention(a, out, lse, 1.0 / hd ** 0.5, rows=list(range(0, len(lens), 17)) + [len(lens) - 1])
    again, lse2 = run_attention(a)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,H,Hk,hd,ps", [(BF, 8, 8, 128, 16), (BF, 24, 1, 64, 8), (F32, 6, 2, 80, 5), (BF, 9, 1, 256, 1)])
@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 7], [64, 63, 1, 0, 17, 33, 2, 0], [0, 128, 127, 65] * 7])
def test_attention_short_streams_few(dtype, H, Hk, hd, ps, lens):
    """So few and short that every stream may have a block of its own, empty sequences among them."""
    a = make_attention(lens, H, Hk, hd, ps, dtype, "token", seed=13)
    out, lse = run_attention(a)
    check_attention(a, out, lse, 1.0 / hd ** 0.5)
    again, lse2 = run_attention(a)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,lens,H,Hk,hd,order,tile", [
    (BF, [4000, 6500, 9000, 1, 0, 5555] * 8, 16, 8, 128, "token", 16),
    (BF, [17000, 33, 9111, 20001] * 12, 16, 4, 64, "head", 32),
    (F32, [2100, 7, 3333, 1500] * 20, 8, 8, 64, "token", 16),
    (BF, [1000 + 7 * i for i in range(300)], 16, 2, 128, "token", 16),   # more lengths than one count covers
])
def test_attention_large_calls(dtype, lens, H, Hk, hd, order, tile):
    """Calls with long pieces, whose joins the pieces name: whole streams and shared ones; the same bits every
    time."""
    a = make_attention(lens, H, Hk, hd, 16, dtype, order, seed=11)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sum(-(-n // tile) for n in lens) * Hk >= 2 * sms * 192   # else a small call
    out, lse = run_attention(a)
    check_attention(a, out, lse, 1.0 / hd ** 0.5, rows=range(0, len(lens), max(1, len(lens) // 12)))
    for _ in range(5):
        again, lse2 = run_attention(a)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_attention_same_bits_and_other_stream():
    a = make_attention([700, 3, 0, 5000, 64], 16, 4, 128, 16, BF, "token", seed=3)
    out, lse = run_attention(a)
    for s in (None, torch.cuda.Stream()):
        again, lse2 = run_attention(a, stream=s)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_strided_and_in_place(dtype):
    """q a slice of the fused projection's rows, out written over it; and q broadcast over the batch."""
    H, Hk, hd = 8, 2, 128
    lens = [50, 700, 0, 16]
    a = make_attention(lens, H, Hk, hd, 16, dtype, "token", seed=4)
    y = randn((4, (H + 2 * Hk) * hd), dtype, 5)
    keep = y.clone()
    q = y[:, :H * hd].unflatten(1, (H, hd))
    a["q"] = q.clone()
    run_attention(a, q=q, out=q)
    check_attention(a, q, None, 1.0 / hd ** 0.5)
    assert torch.equal(y[:, H * hd:], keep[:, H * hd:])
    one = randn((1, 1, hd), dtype, 6).expand(4, H, hd)
    a["q"] = one.clone()
    out, lse = run_attention(a, q=one)
    check_attention(a, out, lse, 1.0 / hd ** 0.5)
    # an odd row stride
    odd = torch.zeros((4, H * hd + 1), dtype=dtype, device="cuda")[:, 1:].unflatten(1, (H, hd))
    odd.copy_(a["q"])
    out2, _ = run_attention(a, q=odd, out=odd)
    check_attention(a, out2, None, 1.0 / hd ** 0.5)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attention_scales(scale):
    a = make_attention([33, 500], 8, 2, 64, 16, BF, "token", seed=6, scale_q=0.5)
    out, _ = run_attention(a, with_lse=False, scale=scale)
    check_attention(a, out, None, float(np.float32(scale)))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_large_scores(dtype):
    """Scores far above fp32's exponential range: only the maximum matters."""
    a = make_attention([1, 40, 2000], 8, 2, 64, 16, dtype, "token", seed=7, scale_q=400.0)
    out, lse = run_attention(a, with_lse=False)
    check_attention(a, out, None, 0.125)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_infinite_and_nan_scores(dtype):
    """Scores of -inf drop out, a row of nothing but -inf gives 0 and lse -inf, a NaN stays within its sequence."""
    lens = [20, 700, 40, 33]
    H, Hk, hd, ps = 4, 1, 64, 16
    a = make_attention(lens, H, Hk, hd, ps, dtype, "token", seed=8)
    a["q"][:, :, 0] = 1.0
    kc = a["cache"].k

    def put(b, j, value):
        page = int(a["tables"][b, j // ps])
        kc[page, j % ps, 0, 0] = value
        a["k"][b][j, 0, 0] = value

    for j in range(lens[0]):
        put(0, j, float("-inf"))
    for j in list(range(0, 400)) + [650]:
        put(1, j, float("-inf"))
    put(2, 39, float("nan"))
    out, lse = run_attention(a)
    assert torch.all(out[0] == 0) and torch.all(torch.isneginf(lse[0]))
    assert torch.all(torch.isnan(out[2]))
    keep = [j for j in range(700) if not (j < 400 or j == 650)]
    a["k"][1], a["v"][1] = a["k"][1][keep], a["v"][1][keep]
    a["lens"][1] = len(keep)
    check_attention(a, out, lse, 0.125, rows=[1, 3])


@pytest.mark.parametrize("dtype,H", [(BF, 8), (F32, 8)])
def test_attention_bad_lengths_and_pages(dtype, H):
    lens = [100, 37, 64, 900, 12, 0]
    hd = 64
    a = make_attention(lens, H, 2, hd, 16, dtype, "token", seed=9)
    a["lengths"][0] = -1
    a["lengths"][2] = a["tables"].shape[1] * 16 + 1
    a["tables"][1, 2] = a["cache"].k.shape[0]      # one past the cache, on the sequence's last page
    a["tables"][3, 30] = -1                        # inside a context that CTAs share
    out, lse = run_attention(a)
    assert lk.lora_get_device_status() == lk.DEV_BAD_LENGTH | lk.DEV_BAD_PAGE
    for b in (0, 1, 2, 3):
        assert torch.all(torch.isnan(out[b])) and torch.all(torch.isnan(lse[b])), b
    check_attention(a, out, lse, 1.0 / hd ** 0.5, rows=[4, 5])


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements: pages near its end."""
    ps, Hk, hd, H = 16, 8, 128, 16
    num_pages = 2 ** 31 // (ps * Hk * hd) + 100
    kc = torch.zeros((num_pages, ps, Hk, hd), dtype=BF, device="cuda")
    vc = torch.zeros((num_pages, ps, Hk, hd), dtype=BF, device="cuda")
    n = 90
    ids = [num_pages - 1, 5, num_pages - 7, num_pages - 90, 131073 % num_pages, num_pages - 2]
    tables = torch.tensor([ids], dtype=torch.int32, device="cuda")
    k, v = randn((n, Hk, hd), BF, 1), randn((n, Hk, hd), BF, 2)
    rows = torch.tensor([ids[j // ps] * ps + j % ps for j in range(n)], dtype=torch.int32, device="cuda")
    cache = lk.KVCache(kc, vc)
    lk.lora_rope_append(lk.RopeProblem(k=k, v=v, cache=cache, cache_rows=rows))
    a = dict(q=randn((1, H, hd), BF, 3), k=[k], v=[v], cache=cache, lens=[n], tables=tables,
             lengths=torch.tensor([n], dtype=torch.int32, device="cuda"))
    out, lse = run_attention(a)
    check_attention(a, out, lse, 1.0 / hd ** 0.5)
    lk.lora_kv_copy_pages(lk.KVCaches([cache]), [ids[0], ids[2]], [num_pages - 20, 3])
    assert torch.equal(kc[num_pages - 20], kc[ids[0]]) and torch.equal(vc[3], vc[ids[2]])


def test_attention_workspace_and_argument_refusals():
    a = make_attention([50], 8, 2, 64, 16, BF, "token")
    out = torch.empty_like(a["q"])
    prob = lk.AttentionProblem(q=a["q"], out=out, cache=a["cache"], block_tables=a["tables"], lengths=a["lengths"])
    need = lk.lora_attention_workspace_bytes(prob)
    ws = lk.new_attention_workspace(prob)
    for bad, code in ((None, 8), (ws.view(torch.uint8)[:need - 1], 8), (ws[1:], 8 if ws.nbytes - 4 < need else 7)):
        with pytest.raises(lk.LoraError) as e:
            lk.lora_paged_attention(prob, bad)
        assert e.value.status == code
    with pytest.raises(ValueError):
        lk.AttentionProblem(q=a["q"].float(), out=out, cache=a["cache"], block_tables=a["tables"],
                            lengths=a["lengths"])
    with pytest.raises(ValueError):
        lk.AttentionProblem(q=a["q"], out=out, cache=a["cache"], block_tables=a["tables"].long(),
                            lengths=a["lengths"])
    with pytest.raises(ValueError):
        lk.AttentionProblem(q=a["q"], out=out, cache=a["cache"], block_tables=a["tables"].cpu(),
                            lengths=a["lengths"])
    with pytest.raises(lk.LoraError) as e:      # 5 query heads over 2 key/value heads
        q5 = torch.empty((1, 5, 64), dtype=BF, device="cuda")
        p5 = lk.AttentionProblem(q=q5, out=torch.empty_like(q5), cache=a["cache"], block_tables=a["tables"],
                                 lengths=a["lengths"])
        lk.lora_paged_attention(p5, ws)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        lk.KVCache(a["cache"].k, a["cache"].v.transpose(1, 2))
    empty = a["q"][:0]
    none = lk.AttentionProblem(q=empty, out=out[:0], cache=a["cache"], block_tables=a["tables"][:0],
                               lengths=a["lengths"][:0])
    lk.lora_paged_attention(none, ws)
    assert lk.lora_last_call_path() == (0, 0)


# ------------------------------------------------------------------ pages --

@pytest.mark.parametrize("dtype,ps,heads,hd,order,layers,pages,n", [
    (BF, 16, 8, 128, "token", 3, 40, 17),
    (BF, 16, 8, 128, "head", 2, 40, 1),
    (BF, 24, 2, 80, "side", 2, 30, 9),
    (BF, 5, 3, 33, "token", 2, 20, 6),       # 2-byte units
    (BF, 4, 2, 64, "gap", 2, 20, 6),
    (F32, 3, 2, 7, "gap", 1, 20, 6),
    (F32, 16, 1, 64, "token", 70, 12, 5),    # more layers than one launch takes
    (BF, 1, 1, 8, "token", 1, 5000, 2300),   # more pages than one launch takes
    (F32, 1, 4, 6, "head", 1, 7, 1),
])
def test_copy_pages(dtype, ps, heads, hd, order, layers, pages, n):
    rng = np.random.default_rng(n)
    ids = rng.permutation(pages)
    src, dst = ids[rng.integers(0, max(1, n // 2), size=n)], ids[n:2 * n]
    it = torch.int16 if dtype == BF else torch.int32
    caches, want = [], []
    for i in range(layers):
        for t in (kv := pool(pages, ps, heads, hd, dtype, order)):
            # any bits at all, NaN payloads among them
            t.view(it).copy_(torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, size=tuple(t.shape))).to(it))
        caches.append(lk.KVCache(*kv))
        for t in kv:
            w = t.view(it).clone()
            w[torch.from_numpy(dst).cuda()] = w[torch.from_numpy(src).cuda()]
            want.append(w)
    lk.lora_kv_copy_pages(lk.KVCaches(caches), src, dst)
    got = [t.view(it) for c in caches for t in (c.k, c.v)]
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    if order == "gap":     # the gaps are not touched
        whole = caches[0].k.as_strided((pages, ps, heads, 3), caches[0].k.stride(), hd)
        assert torch.all(torch.isnan(whole))


def test_copy_pages_refusals():
    c = lk.KVCaches([lk.KVCache(*pool(30, 4, 2, 8, BF, "token", fill=1.0))])
    long_src, long_dst = list(range(20)), [20] * 19 + [21]
    for src, dst in (([0], [0]), ([0, 1], [1, 2]), ([0, 0], [3, 3]), ([30], [0]), ([0], [-1]), ([0], [30]),
                     (long_src[:9], long_dst[:9]), (long_src[:18], [0] + list(range(20, 30)) + [19] * 7)):
        with pytest.raises(lk.LoraError) as e:
            lk.lora_kv_copy_pages(c, src, dst)
        assert e.value.status == 2, (src, dst)
    two = lk.KVCaches([c.layers[0], lk.KVCache(*pool(31, 4, 2, 8, BF, "token", fill=1.0))])
    with pytest.raises(lk.LoraError) as e:
        lk.lora_kv_copy_pages(two, [0], [1])
    assert e.value.status == 2
    with pytest.raises(ValueError):
        lk.lora_kv_copy_pages(c, [0, 1], [2])
    lk.lora_kv_copy_pages(c, [], [])
    assert lk.lora_last_call_path() == (0, 0)
