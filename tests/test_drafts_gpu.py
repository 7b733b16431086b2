"""The verification of drafted tokens on the GPU (4-bit base projection, tree
attention, kept rows) against definitions in 64 bits, at the sizes, layouts and
masks where they can go wrong.

Bounds, with e = 2^-24 (fp32's half step at 1) and h = 2^-8 (bf16's, relative):
  tree   a score is a sum of head_dim products, off by (head_dim + 8) e times
         scale sum |q k|, and twice that where the tensor cores cut sums off
         instead of rounding; a probability is off by as much relatively, and by
         2^-16 as two bf16 terms (the first cut off: 2^-7 of it is left, the
         second rounded: 2^-9 of that).  The output is a sum of len products
         over a sum of len: (2 len + 16) e, twice that likewise.  Times the
         weighted mean of |v|.
  q4     a sum of in products: lanes and instructions share it out, no term goes
         through more than in / 4 + 32 sums (16 inputs an instruction, three
         cuts each; a lane of 32 in the generic kernel; one sum a group), each
         off by 2 e of at most sum |w x|; the delta's factors A x likewise, then
         R more, and u enters as two bf16 terms at 2^-16.
  rounding   bf16 results: h |ref| on top; all also 2^-126 (subnormals).
"""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: E}
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


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


def ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ------------------------------------------------------- 4-bit projection --

def codes_of(q, n):
    q = q.cpu().numpy()
    return np.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)[:, :n].astype(np.float64)


class Q4Case:
    def __init__(self, T, n, outs, group, R, dtype, counts, S=4, zeros=True, bias=False, ranks=False, seed=0,
                 x_gap=0, y_gap=0, q_gap=0, extra_zero=False):
        rng = np.random.default_rng(seed)
        self.n, self.outs, self.R, self.dtype, self.T, self.group = n, outs, R, dtype, T, group
        O, groups = sum(outs), -(-n // group)
        qb = -(-n // 2)
        q = torch.from_numpy(rng.integers(0, 256, size=(O, qb + q_gap), dtype=np.uint8)).cuda()
        self.q = q[:, :qb]
        self.scales = ((torch.rand((O, groups), generator=torch.Generator().manual_seed(seed)) + 0.5) *
                       (0.2 / n ** 0.5)).to(dtype).cuda()
        self.zeros = None
        if zeros:
            z = rng.integers(0, 256 if extra_zero else 16, size=(O, groups), dtype=np.uint8)
            self.zeros = torch.from_numpy(z).cuda()
        self.a = randn((S, len(outs) * R, n), dtype, seed + 1, n ** -0.5)
        self.b = randn((S, O, R), dtype, seed + 2, 0.3)
        self.slot_ranks = None
        if ranks:
            r = rng.integers(0, R + 1, size=S)
            self.slot_ranks = ints(r)
            for s in range(S):
                self.b[s, :, r[s]:] = 0
                for j in range(len(outs)):
                    self.a[s, j * R + r[s]:(j + 1) * R] = 0
        x = randn((T, n + x_gap), dtype, seed + 3)
        self.x = x[:, :n]
        y = torch.full((T + 2, O + y_gap), NAN, dtype=dtype, device="cuda")
        self.whole_y, self.y = y, y[:T, :O]
        self.bias = randn((S, O), dtype, seed + 4) if bias else None
        # counts: rows of slot 0, 1, ...; the others are base rows
        self.ids = [s for s, c in enumerate(counts) if c is not None]
        self.offs = np.cumsum([0] + [c for c in counts if c is not None]).astype(np.int32)
        self.end = int(self.offs[-1])
        p = lk.fused_problem(self.x, self.a, self.b, self.y, outs)
        if bias:
            off = 0
            for s, o in zip(p.slices, outs):
                s.bias, s.bias_slot_stride, s.bias_offset = self.bias, O, off
                off += o
        p.slot_ranks = self.slot_ranks
        self.problem = p
        cut = np.cumsum([0] + outs)
        self.weights = [lk.Q4Weight(self.q[i:j], self.scales[i:j], group,
                                    zeros=None if self.zeros is None else self.zeros[i:j])
                        for i, j in zip(cut[:-1], cut[1:])]
        self.routing = lk.Routing(ints(self.ids), ints(self.offs), len(self.ids), self.end)
        self.call = lk.BaseQ4Problem(p, self.routing, self.weights)
        self.workspace = lk.new_workspace(p, self.end)

    def run(self, **kw):
        lk.lora_base_q4_apply(self.call, self.workspace, **kw)
        return self.y

    def reference(self):
        """(y, sum of magnitudes of the base product, of the delta) in 64 bits."""
        of = np.arange(self.n) // self.group
        zero = 8.0 if self.zeros is None else f64(self.zeros)[:, of]
        w = (codes_of(self.q, self.n) - zero) * f64(self.scales)[:, of]
        x = f64(self.x)
        y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
        dmag = np.zeros_like(y)
        a, b = f64(self.a), f64(self.b)
        for s, lo, hi in zip(self.ids, self.offs[:-1], self.offs[1:]):
            col = 0
            for j, o in enumerate(self.outs):
                aj, bj = a[s, j * self.R:(j + 1) * self.R], b[s, col:col + o]
                y[lo:hi, col:col + o] += x[lo:hi] @ aj.T @ bj.T
                dmag[lo:hi, col:col + o] += np.abs(x[lo:hi]) @ np.abs(aj).T @ np.abs(bj).T
                col += o
            if self.bias is not None:
                y[lo:hi] += f64(self.bias)[s]
                mag[lo:hi] += np.abs(f64(self.bias)[s])
        return y, mag, dmag

    def check(self):
        ref, mag, dmag = self.reference()
        depth = 2 * E * (self.n / 4 + 32)
        tol = depth * mag + (depth + 2 * E * (self.R + 8) + 2.0 ** -16) * dmag + ROUND[self.dtype] * np.abs(ref) + 2.0 ** -126
        err = np.abs(f64(self.y) - ref)
        assert np.all(err <= tol), (float(np.nanmax(err - tol)), np.argwhere(~(err <= tol))[:4])
        # nothing but y's rows and columns is written
        whole = self.whole_y
        assert torch.isnan(whole[self.T:]).all() and torch.isnan(whole[:, sum(self.outs):]).all()


Q4_CASES = [
    # T, in, outs, group, R, dtype, rows of slots 0, 1, ...
    (1, 256, [64], 64, 16, BF, [1]),
    (1, 4096, [96, 32, 32], 128, 16, BF, [None, 1]),
    (2, 64, [8], 32, 16, BF, [1]),
    (3, 128, [24, 8], 128, 32, BF, [1, 0, 2]),
    (5, 512, [136], 32, 64, BF, [2, None, 2]),
    (7, 320, [72, 16, 8], 64, 128, BF, []),              # base rows alone
    (8, 1024, [256, 128], 1024, 16, BF, [8]),            # a group a row
    (9, 1024, [256], 256, 16, BF, [3, 3, 1]),
    (16, 256, [128], 64, 16, BF, [5, 5]),
    (17, 256, [144], 64, 16, BF, [0, 17]),
    (31, 384, [200], 128, 32, BF, [10, 0, 3, 9]),
    (33, 192, [128, 64], 96, 16, BF, [30, 3]),
    (64, 256, [264], 32, 16, BF, [20, 1, 40]),
    (65, 512, [128], 128, 64, BF, [64]),
    (100, 576, [120, 24, 24], 64, 16, BF, [50, 30]),
    (129, 256, [128], 64, 16, BF, [100, 29]),
    (300, 512, [256, 40], 128, 128, BF, [200, 50, 7]),   # long groups
    (4, 256, [64], 64, 8, BF, [2, 1]),                   # a rank that the tensor-core shrink does not take
    (4, 250, [63], 64, 16, BF, [2, 1]),                  # widths that the fast path does not take
    (4, 256, [61], 64, 16, BF, [2, 1]),
    (4, 256, [64], 40, 16, BF, [2, 1]),                  # a group that is no multiple of 32
    (3, 101, [7, 5], 13, 3, BF, [1, 1]),
    (1, 1, [1], 1, 1, F32, [1]),
    (1, 256, [64], 64, 16, F32, [1]),
    (9, 333, [50, 21], 40, 8, F32, [2, 5]),
    (20, 128, [130], 128, 16, F32, [3, 3, 3]),
]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("case", Q4_CASES, ids=lambda c: "-".join(str(x) for x in c).replace("torch.", "").replace(" ", ""))
def test_q4(case, zeros):
    c = Q4Case(*case, zeros=zeros)
    c.run()
    n, group, dtype = case[1], case[3], case[5]
    fast = dtype == BF and n % 32 == 0 and (group % 32 == 0 or group >= n)
    path = lk.lora_last_call_path()[0]
    assert bool(path & (lk.PATH_MMA_Q4 | lk.PATH_TC_Q4)) == fast and bool(path & lk.PATH_GENERIC_Q4) == (not fast)
    c.check()
    first = c.y.clone()
    c.run()
    assert torch.equal(first, c.y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,R", [(1, 16), (6, 64), (40, 16), (140, 64)])
def test_q4_bias_ranks_and_gaps(dtype, T, R):
    c = Q4Case(T, 512, [64, 128], 64, R, dtype, [T // 3, 0, T - T // 3], bias=True, ranks=True, x_gap=8, y_gap=8, q_gap=16)
    c.run()
    c.check()
    c = Q4Case(T, 512, [64, 128], 64, R, dtype, [T], x_gap=1, y_gap=3, q_gap=1, seed=5)   # nothing on a boundary
    c.run()
    c.check()


def test_q4_zeros_of_any_byte():
    """A zero past 15 (packed as q + 1, say) is a number like any other."""
    for T, dtype in ((3, BF), (90, BF), (3, F32)):
        c = Q4Case(T, 256, [128], 64, 16, dtype, [T], extra_zero=True)
        c.run()
        c.check()


@pytest.mark.parametrize("T", [1, 5, 20, 80, 130])
def test_q4_extremes(T):
    """Every code 0 or 15, all inputs equal: no sum of a group may pass a narrow type's range."""
    c = Q4Case(T, 2048, [64], 2048, 16, BF, [], zeros=False)
    for byte in (0x00, 0xFF):
        c.q.fill_(byte)
        c.x.fill_(3.0)
        c.run()
        c.check()


@pytest.mark.parametrize("T", [1, 3, 8, 9, 16])
@pytest.mark.parametrize("n,group", [(96, 32), (320, 64), (512, 128), (1024, 1024)])
def test_q4_many_outputs(T, n, group):
    """More tiles of outputs than CTAs: few rows that walk them, odd ends, a slice that ends inside a tile."""
    outs = [9800, 40, 233]
    c = Q4Case(T, n, outs, group, 32, BF, [T // 3, None, T - T // 3 - T // 4], bias=True, ranks=True, x_gap=8, y_gap=7,
               q_gap=16, extra_zero=T == 3)
    c.run()
    assert lk.lora_last_call_path()[0] & lk.PATH_MMA_Q4
    c.check()
    clean = c.y.clone()
    if T > 1:
        c.x[T - 1, n - 1] = NAN
        c.x[0, 3] = float("inf")
        c.run()
        assert torch.equal(c.y[1:T - 1], clean[1:T - 1])
        assert torch.isnan(c.y[T - 1]).all() and torch.isfinite(c.y[0]).sum() < 9800 // 2


@pytest.mark.parametrize("T,n,group,outs,R", [
    (300, 192, 64, [4000, 40], 16), (700, 640, 128, [2056, 1000, 77], 64), (513, 224, 192, [4096], 128),
    (512, 96, 96, [5000], 8), (130, 320, 64, [16000], 256), (48, 256, 128, [9900, 300], 24), (401, 128, 128, [4130], 3)])
@pytest.mark.parametrize("zeros", [False, True])
def test_q4_many_rows(T, n, group, outs, R, zeros):
    """Enough work for the kernel on tcgen05: odd ends, groups of one and two blocks, runs of rows within and across
    tiles, base rows between a tile's runs and the end."""
    counts = [T // 5, 1, None, 0, T // 10, T // 2 - 1]
    c = Q4Case(T, n, outs, group, R, BF, counts, S=6, zeros=zeros, bias=True, ranks=R >= 16, x_gap=8, y_gap=3,
               q_gap=16, extra_zero=zeros and T == 300)
    c.run()
    assert lk.lora_last_call_path()[0] & lk.PATH_TC_Q4
    c.check()
    clean = c.y.clone()
    c.run()
    assert torch.equal(c.y, clean)
    # what a slot or a row holds stays with its own rows
    c.x[T - 1, n - 1] = NAN
    c.x[2, 1] = float("inf")
    c.b[1] = NAN
    c.run()
    row = int(c.offs[1])
    read = c.slot_ranks is None or int(c.slot_ranks[1]) > 0   # of a slot of rank 0 nothing is read
    others = [t for t in range(T) if t not in (2, T - 1) and not (read and t == row)]
    assert torch.equal(c.y[others], clean[others])
    assert torch.isnan(c.y[T - 1]).all() and (not read or torch.isnan(c.y[row]).all())


def test_q4_many_rows_streams_graph_and_bad_routing():
    c = Q4Case(300, 256, [4000, 64], 64, 16, BF, [100, 0, 90])
    want = c.run().clone()
    assert lk.lora_last_call_path()[0] & lk.PATH_TC_Q4
    c.y.fill_(NAN)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    assert torch.equal(c.y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.y.fill_(NAN)
    c.x.copy_(randn(c.x.shape, BF, 98))
    g.replay()
    c.check()
    c.y.fill_(NAN)
    c.routing.lora_ids.fill_(77)
    c.run()
    assert lk.lora_get_device_status() & lk.DEV_BAD_SLOT
    assert torch.isnan(c.y).all()


def test_q4_row_with_infinity_and_nan():
    """Inputs that are infinite or NaN stay with their own row."""
    for T in (4, 40, 140):
        c = Q4Case(T, 512, [128], 64, 16, BF, [T // 2])
        clean = c.run().clone()
        c.x[1, 7] = float("inf")
        c.x[T - 1, 300] = NAN
        c.run()
        others = [t for t in range(T) if t not in (1, T - 1)]
        assert torch.equal(c.y[others], clean[others])
        assert not torch.isfinite(c.y[1]).any() or torch.isfinite(c.y[1]).sum() < 128
        assert torch.isnan(c.y[T - 1]).all()


def test_q4_streams_and_graph():
    c = Q4Case(12, 1024, [256, 64], 128, 16, BF, [5, 0, 4])
    want = c.run().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.y.fill_(NAN)
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    s.synchronize()
    assert torch.equal(c.y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.y.fill_(NAN)
    g.replay()
    assert torch.equal(c.y, want)
    c.x.copy_(randn(c.x.shape, BF, 99))
    g.replay()
    c.check()


@pytest.mark.parametrize("T,outs", [(2, [512]), (12, [512, 96]), (300, [4000, 40])])
def test_q4_two_calls_at_once(T, outs):
    """Two calls in flight on two streams, each with its workspace, and two captured graphs replayed likewise."""
    cs = [Q4Case(T, 512, outs, 64, 16, BF, [T // 2, T - T // 2 - 1], seed=i) for i in range(2)]
    want = [c.run().clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    graphs = []
    for c in cs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.run()
    for replay in (False, True):
        for c in cs:
            c.y.fill_(NAN)
        torch.cuda.synchronize()
        for _ in range(5):
            for c, s, g in zip(cs, streams, graphs):
                with torch.cuda.stream(s):
                    g.replay() if replay else c.run()
        torch.cuda.synchronize()
        for c, w in zip(cs, want):
            assert torch.equal(c.y, w)


def test_q4_bad_routing_writes_nothing():
    for dtype in (BF, F32):
        c = Q4Case(9, 256, [64], 64, 16, dtype, [4, 5])
        c.run()
        c.y.fill_(NAN)
        c.routing.lora_ids.fill_(77)
        c.run()
        assert lk.lora_get_device_status() & lk.DEV_BAD_SLOT
        assert torch.isnan(c.y).all()


# --------------------------------------------------------- tree attention --

def tree_case(rows, ctx, H, Hk, hd, ps, dtype, order="token", masks="tree", pad=0, words=None, seed=0, fill=NAN):
    """Sequences with `rows` drafted tokens behind `ctx` cached ones, pages in a random order; every cell of the
    cache that no sequence holds is `fill`."""
    rng = np.random.default_rng(seed)
    lens = [c + n for c, n in zip(ctx, rows)]
    need = [-(-n // ps) for n in lens]
    num_pages = sum(need) + 2
    ids = rng.permutation(num_pages)
    tables = np.full((len(rows), max(1, max(need)) + 1), 10 ** 9, dtype=np.int32)   # nonsense behind the last page
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
    if order == "token":
        kc, vc = (torch.full((num_pages, ps, Hk, hd), fill, dtype=dtype, device="cuda") for _ in range(2))
    elif order == "head":
        kc, vc = (torch.full((num_pages, Hk, ps, hd), fill, dtype=dtype, device="cuda").transpose(1, 2) for _ in range(2))
    elif order == "side":     # K and V side by side within a token
        both = torch.full((num_pages, ps, 2, Hk, hd), fill, dtype=dtype, device="cuda")
        kc, vc = both[:, :, 0], both[:, :, 1]
    else:                     # rows with a gap of 3 elements: nothing on a 16-byte boundary
        kc, vc = (torch.full((num_pages, ps, Hk, hd + 3), fill, dtype=dtype, device="cuda")[..., :hd] for _ in range(2))
    k, v = [], []
    for b, n in enumerate(lens):
        kb, vb = randn((n, Hk, hd), dtype, seed + 10 * b + 1), randn((n, Hk, hd), dtype, seed + 10 * b + 2)
        pos = torch.arange(n)
        page = torch.from_numpy(tables[b].astype(np.int64))[pos // ps].cuda()
        kc[page, pos.cuda() % ps] = kb
        vc[page, pos.cuda() % ps] = vb
        k.append(kb)
        v.append(vb)
    N = sum(rows) + pad
    W = words or max(1, -(-max(rows + [1]) // 64))
    m = np.zeros((N, W), dtype=np.uint64)
    sees = []
    at = 0
    for b, n in enumerate(rows):
        if masks == "tree":
            par = [-1] + [int(rng.integers(-1, i)) for i in range(1, n)]
            m[at:at + n] = lk.lora_build_tree(par[:n], W)["masks"]
        elif masks == "random":     # no tree at all, bits of tokens that are not there among them
            m[at:at + n] = rng.integers(0, 2 ** 64, size=(n, W), dtype=np.uint64) & rng.integers(0, 2 ** 64, size=(n, W), dtype=np.uint64)
            m[at:at + n:3] = 0
        bits = np.unpackbits(m[at:at + n].view(np.uint8).reshape(n, 8 * W), axis=1, bitorder="little")[:, :n].astype(bool)
        if masks is None:
            bits = np.tril(np.ones((n, n), dtype=bool))
        sees.append(np.concatenate((np.ones((n, ctx[b]), dtype=bool), bits), 1))
        at += n
    q = randn((N, H, hd), dtype, seed + 7, 1.5)
    return dict(q=q, k=k, v=v, cache=lk.KVCache(kc, vc), tables=ints(tables), lengths=ints(lens),
                offsets=ints(np.cumsum([0] + rows)), rows=rows, ctx=ctx, sees=sees, N=N, H=H, Hk=Hk, hd=hd,
                masks=None if masks is None else torch.from_numpy(m.view(np.int64)).cuda(), dtype=dtype)


def run_tree(a, q=None, out=None, stream=None, scale=None):
    q = a["q"] if q is None else q
    out = torch.full((a["N"], a["H"], a["hd"]), NAN, dtype=a["dtype"], device="cuda") if out is None else out
    lse = torch.full((a["N"], a["H"]), NAN, device="cuda")
    p = lk.TreeAttentionProblem(q=q, out=out, cache=a["cache"], block_tables=a["tables"], lengths=a["lengths"],
                                row_offsets=a["offsets"], masks=a["masks"], lse=lse, scale=scale)
    ws = lk.new_tree_attention_workspace(p)
    ws.fill_(NAN)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    lk.lora_tree_attention(p, ws, stream=stream)
    if stream is not None:
        stream.synchronize()
    return out, lse


def check_tree(a, out, lse, scale=None, skip=(), seqs=None):
    G, hd = a["H"] // a["Hk"], a["hd"]
    scale = hd ** -0.5 if scale is None else scale
    o64, l64, q64 = f64(out), f64(lse) if lse is not None else None, f64(a["q"])
    tc = a["dtype"] == BF
    at = 0
    for b, n in enumerate(a["rows"]):
        lo, at = at, at + n
        if b in skip or (seqs is not None and b not in seqs):
            continue
        if n == 0:
            continue
        k, v = f64(a["k"][b]), f64(a["v"][b])
        L = k.shape[0]
        for h in range(a["H"]):
            kk, vv = k[:, h // G], v[:, h // G]
            z = scale * (q64[lo:at, h] @ kk.T)
            zmag = abs(scale) * (np.abs(q64[lo:at, h]) @ np.abs(kk).T)
            z = np.where(a["sees"][b], z, -np.inf)
            top = z.max(1, keepdims=True)
            w = np.exp(z - np.where(np.isinf(top), 0, top))
            s = w.sum(1, keepdims=True)
            p = w / np.where(s == 0, 1, s)
            ref = p @ vv
            serr = (2 if tc else 1) * (hd + 8) * E * np.where(a["sees"][b], zmag, 0).max(1, keepdims=True)
            rel = 2 * serr + (2 if tc else 1) * (2 * L + 16) * E + (2.0 ** -16 if tc else 0)
            tol = rel * (p @ np.abs(vv)) + ROUND[a["dtype"]] * np.abs(ref) + 2.0 ** -126
            err = np.abs(o64[lo:at, h] - ref)
            assert np.all(err <= tol), (b, h, float(np.nanmax(err - tol)), np.argwhere(~(err <= tol))[:3])
            if lse is not None:
                with np.errstate(divide="ignore"):
                    rl = (top + np.log(s))[:, 0]
                got = l64[lo:at, h]
                none = np.isneginf(rl)
                assert np.all(np.isneginf(got[none])) and np.all(o64[lo:at, h][none] == 0)
                ltol = serr[:, 0] + (2 * L + 16 + 4 * np.abs(np.where(none, 0, rl))) * 2 * E
                assert np.all(np.abs(got[~none] - rl[~none]) <= ltol[~none])
    # rows behind the last sequence
    assert torch.isnan(out[at:]).all() and (lse is None or torch.isnan(lse[at:]).all())


RAGGED = ([1, 2, 0, 7, 8, 9, 16, 17, 31, 33, 64, 5, 5, 3, 1], [0, 1, 50, 8, 120, 119, 112, 111, 128, 257, 64, 1000, 0, 13, 127])
TREE_CASES = [
    # dtype, (rows, contexts), H, Hk, hd, page_size, order
    (BF, RAGGED, 8, 2, 128, 16, "token"),
    (BF, RAGGED, 32, 8, 128, 16, "head"),
    (BF, RAGGED, 8, 8, 64, 16, "token"),
    (BF, RAGGED, 14, 2, 64, 24, "side"),      # 7 heads a group
    (BF, RAGGED, 6, 2, 128, 3, "token"),      # pages that are no multiple of anything
    (BF, RAGGED, 16, 1, 80, 8, "head"),
    (BF, RAGGED, 20, 1, 96, 1, "token"),      # 20 heads a group
    (BF, RAGGED, 8, 2, 256, 16, "token"),
    (BF, RAGGED, 6, 2, 200, 64, "head"),
    (BF, RAGGED, 4, 2, 32, 16, "token"),
    (BF, RAGGED, 4, 2, 8, 16, "token"),
    (BF, RAGGED, 4, 2, 33, 16, "token"),      # odd width
    (BF, RAGGED, 4, 2, 64, 16, "gap"),        # rows off 16-byte boundaries
    (F32, RAGGED, 8, 2, 128, 16, "token"),
    (F32, RAGGED, 6, 6, 64, 5, "head"),
    (F32, RAGGED, 4, 2, 256, 16, "side"),
    (F32, RAGGED, 9, 3, 100, 16, "token"),
    (F32, RAGGED, 3, 3, 7, 2, "gap"),
    (BF, ([1], [0]), 4, 2, 64, 16, "token"),
    (BF, ([6], [517]), 32, 8, 128, 16, "token"),
    (BF, ([60], [9000]), 8, 2, 128, 32, "token"),             # one context over many CTAs
    (BF, ([200, 3], [300, 2000]), 8, 2, 128, 16, "token"),    # several words a row, several chunks a stream
    (F32, ([100, 3], [300, 2000]), 4, 2, 64, 16, "token"),
    (F32, ([9], [5000]), 4, 1, 128, 16, "token"),
    (BF, ([4] * 150, [30 + i for i in range(150)]), 8, 2, 64, 16, "token"),   # more streams than CTAs
    (BF, ([13, 26, 5, 9] * 6, [700, 1500, 128, 2048] * 6), 8, 4, 128, 16, "head"),
]


@pytest.mark.parametrize("masks", ["tree", None])
@pytest.mark.parametrize("case", TREE_CASES, ids=lambda c: "%s-%dseq-%d-%d-%d-%d-%s" % (str(c[0])[6:], len(c[1][0]), *c[2:]))
def test_tree(case, masks):
    dtype, (rows, ctx), H, Hk, hd, ps, order = case
    a = tree_case(list(rows), list(ctx), H, Hk, hd, ps, dtype, order, masks, pad=3)
    out, lse = run_tree(a)
    tc = dtype == BF and hd % 8 == 0 and order != "gap"
    assert lk.lora_last_call_path()[0] & ~lk.PATH_JOIN == (lk.PATH_TC_TREE if tc else lk.PATH_GENERIC_TREE)
    seqs = None if len(rows) < 30 else list(range(0, len(rows), 13)) + [len(rows) - 1]
    check_tree(a, out, lse, seqs=seqs)
    again, lse2 = run_tree(a)
    n = sum(rows)
    assert torch.equal(out[:n], again[:n]) and torch.equal(lse[:n], lse2[:n])


@pytest.mark.parametrize("dtype,hd", [(BF, 128), (BF, 64), (BF, 256), (F32, 64)])
def test_tree_masks_of_any_kind(dtype, hd):
    """Masks that are no trees, rows that see nothing (of sequences without a context), bits of tokens that the
    sequence does not have."""
    rows, ctx = [5, 70, 130, 1, 2, 33], [0, 0, 31, 0, 129, 1]
    a = tree_case(rows, ctx, 8, 2, hd, 16, dtype, masks="random", words=4, pad=2, seed=3)
    out, lse = run_tree(a)
    check_tree(a, out, lse)
    assert torch.isneginf(lse[0]).all() and (out[0] == 0).all()


@pytest.mark.parametrize("dtype,hd", [(BF, 128), (BF, 64), (BF, 256), (F32, 64), (BF, 33)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), NAN, 3e38])
def test_tree_unseen_values_have_no_part(dtype, hd, value):
    """Keys and values of other branches that are infinite, NaN or huge: the rows that do not see them are the
    same bit for bit; a row that sees such a value has it."""
    rows, ctx = [40, 9, 3], [100, 0, 500]
    a = tree_case(rows, ctx, 4, 2, hd, 16, dtype, seed=4)
    clean, _ = run_tree(a)
    kc, vc = a["cache"].k, a["cache"].v
    tables = a["tables"].cpu().numpy()
    at = 0
    for b, (n, c) in enumerate(zip(rows, ctx)):
        tok = n - 2                                    # this drafted token's V (and the last one's K and V)
        touched = {}
        for t, both in ((tok, False), (n - 1, True)):
            page, off = int(tables[b, (c + t) // 16]), (c + t) % 16
            touched[t] = (page, off, kc[page, off].clone(), vc[page, off].clone())
            vc[page, off] = value
            if both:
                kc[page, off] = value
        out, _ = run_tree(a)
        blind = [i for i in range(n) if not a["sees"][b][i, c + tok] and not a["sees"][b][i, c + n - 1]]
        assert blind and torch.equal(out[at:at + n][blind], clean[at:at + n][blind])
        sees = [i for i in range(n) if a["sees"][b][i, c + tok] and not a["sees"][b][i, c + n - 1]]
        if not np.isfinite(value):
            got = out[at:at + n][sees]
            assert sees and (torch.isnan(got).all() if value != value else (got == value).all())
        for page, off, k0, v0 in touched.values():
            kc[page, off], vc[page, off] = k0, v0
        at += n


def test_tree_in_place_strided_broadcast():
    """q a slice of the fused projection's rows, out written over it; q broadcast over heads."""
    for dtype, hd in ((BF, 128), (BF, 256), (F32, 64)):
        H, Hk = 8, 2
        a = tree_case([9, 30, 2], [300, 64, 0], H, Hk, hd, 16, dtype, seed=5)
        y = randn((a["N"], (H + 2 * Hk) * hd), dtype, 6)
        keep = y.clone()
        q = y[:, :H * hd].unflatten(1, (H, hd))
        a["q"] = q.clone()
        out, lse = run_tree(a, q=q, out=q)
        check_tree(a, out, lse)
        assert torch.equal(y[:, H * hd:], keep[:, H * hd:])
        one = randn((a["N"], 1, hd), dtype, 7).expand(a["N"], H, hd)
        a["q"] = one.clone()
        out, lse = run_tree(a, q=one, scale=-0.3)
        check_tree(a, out, lse, scale=-0.3)
        odd = torch.full((a["N"], H * hd + 1), NAN, dtype=dtype, device="cuda")[:, 1:].unflatten(1, (H, hd))
        run_tree(a, out=odd)
        check_tree(a, odd, None)


def test_tree_equals_paged_attention_for_single_tokens():
    """A chain of one is the framework's decode attention."""
    for dtype in (BF, F32):
        a = tree_case([1] * 6, [0, 5, 127, 128, 900, 40], 8, 2, 128, 16, dtype, masks=None)
        out, lse = run_tree(a)
        check_tree(a, out, lse)
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        p = lk.AttentionProblem(q=a["q"], out=o2, cache=a["cache"], block_tables=a["tables"], lengths=a["lengths"], lse=l2)
        lk.lora_paged_attention(p, lk.new_attention_workspace(p))
        check_tree(a, o2, l2)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_far_offsets(dtype):
    """Pages whose elements lie past 2^31 and 2^32 elements of the cache's start."""
    ps, Hk, hd = 16, 8, 128
    stride = 2 ** 31 // 3 + 8
    base = torch.empty(8 * stride, dtype=dtype, device="cuda")
    kc = base.as_strided((7, ps, Hk, hd), (stride, Hk * hd, hd, 1))
    vc = base[ps * Hk * hd:].as_strided((7, ps, Hk, hd), (stride, Hk * hd, hd, 1))
    a = tree_case([5], [107], 8, Hk, hd, ps, dtype, seed=8)
    order = [6, 0, 5, 1, 4, 2, 3]
    for i, page in enumerate(order):
        kc[page] = a["k"][0][16 * i:16 * i + 16]
        vc[page] = a["v"][0][16 * i:16 * i + 16]
    a["cache"], a["tables"] = lk.KVCache(kc, vc), ints([order])
    out, lse = run_tree(a)
    check_tree(a, out, lse)


def test_tree_bad_lengths_pages_offsets():
    for dtype in (BF, F32):
        rows, ctx = [4, 70, 9, 3], [100, 30, 0, 700]
        a = tree_case(rows, ctx, 8, 2, 64, 16, dtype, words=2)
        first = np.cumsum([0] + rows)
        lengths, tables = a["lengths"].clone(), a["tables"].clone()

        def others_same(bad, flag):
            out, lse = run_tree(a)
            assert lk.lora_get_device_status() == flag
            for b in bad:
                lo, hi = first[b], first[b + 1]
                assert torch.isnan(out[lo:hi]).all() and torch.isnan(lse[lo:hi]).all()
            check_tree(a, out, lse, skip=bad)

        for b, bad_len in ((0, 3), (1, -5), (3, 10 ** 9), (2, 0), (2, -2 ** 31)):
            a["lengths"] = lengths.clone()
            a["lengths"][b] = bad_len
            others_same([b], lk.DEV_BAD_LENGTH)
        a["lengths"] = lengths
        for b, col, page in ((0, 2, -1), (3, 43, 10 ** 6), (3, 0, 2 ** 31 - 1), (1, 6, -2 ** 31)):
            a["tables"] = tables.clone()
            a["tables"][b, col] = page
            others_same([b], lk.DEV_BAD_PAGE)
        a["tables"] = tables
        offsets = a["offsets"].clone()
        for i, v in ((0, -1), (2, 3), (4, 10 ** 6), (4, a["N"] + 1)):
            a["offsets"] = offsets.clone()
            a["offsets"][i] = v
            out, lse = run_tree(a)
            assert lk.lora_get_device_status() == lk.DEV_BAD_OFFSETS
            assert torch.isnan(out).all() and torch.isnan(lse).all()
        a["offsets"] = offsets
        a["masks"] = a["masks"][:, :1].contiguous()      # 64 bits for 70 rows
        others_same([1], lk.DEV_BAD_LENGTH)


def test_tree_streams_graph_and_two_workspaces():
    a = tree_case([26, 9, 40], [900, 3000, 17], 8, 2, 128, 16, BF, seed=9)
    want, wlse = run_tree(a)
    out, lse = run_tree(a, stream=torch.cuda.Stream())
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    o1 = torch.empty_like(want)
    p = lk.TreeAttentionProblem(q=a["q"], out=o1, cache=a["cache"], block_tables=a["tables"], lengths=a["lengths"],
                                row_offsets=a["offsets"], masks=a["masks"])
    ws = lk.new_tree_attention_workspace(p)
    g = torch.cuda.CUDAGraph()
    lk.lora_tree_attention(p, ws)
    with torch.cuda.graph(g):
        lk.lora_tree_attention(p, ws)
    o1.fill_(NAN)
    ws.fill_(NAN)
    g.replay()
    assert torch.equal(o1, want)
    # other lengths, the graph replayed: the lengths are read by the kernels
    a["lengths"].copy_(ints([500 + 26, 3009, 57]))
    a["k"][0], a["v"][0] = None, None
    g.replay()
    fresh, _ = run_tree(a)
    assert torch.equal(o1, fresh)


def test_tree_no_rows_and_no_sequences():
    a = tree_case([2, 3], [5, 6], 4, 2, 64, 16, BF)
    a["offsets"].zero_()
    out, lse = run_tree(a)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    p = lk.TreeAttentionProblem(q=a["q"], out=out, cache=a["cache"], block_tables=a["tables"][:0], lengths=a["lengths"][:0],
                                row_offsets=a["offsets"][:1])
    lk.lora_tree_attention(p, lk.new_tree_attention_workspace(p))
    assert lk.lora_last_call_path() == (0, 0)


# -------------------------------------------------------------- kept rows --

@pytest.mark.parametrize("dtype,Hk,hd,ps,order,layers", [
    (BF, 8, 128, 16, "token", 3), (BF, 8, 128, 16, "head", 70), (BF, 2, 80, 5, "side", 2), (BF, 3, 33, 1, "token", 2),
    (BF, 2, 64, 16, "gap", 2), (F32, 4, 64, 8, "token", 2), (F32, 1, 7, 3, "gap", 1), (BF, 40, 256, 4, "token", 1)])
def test_keep_rows(dtype, Hk, hd, ps, order, layers):
    rng = np.random.default_rng(1)
    rows, ctx = [1, 9, 0, 26, 40, 3, 64], [0, 5, 9, 131, 15, 16, 1]
    cases = [tree_case(rows, ctx, Hk, Hk, hd, ps, dtype, order, seed=20 + i, fill=5.0) for i in range(min(layers, 3))]
    a = cases[0]
    caches = [c["cache"] for c in cases]
    caches = [caches[i % len(caches)] for i in range(3)][:layers] if layers <= 3 else [
        lk.KVCache(a["cache"].k.clone(memory_format=torch.preserve_format), a["cache"].v.clone(memory_format=torch.preserve_format))
        for _ in range(layers)]
    K = 30
    path = np.full((len(rows), K), -1, dtype=np.int32)
    paths = []
    for b, n in enumerate(rows):
        m = [1, 3, 0, 8, 30, 0, 20][b]
        keep = sorted(rng.choice(n, size=m, replace=False).tolist()) if m else []
        if b == 4:
            keep = list(range(10, 40))     # every row moved onto rows that are moved themselves
        path[b, :m] = keep
        if m + 1 < K:
            path[b, m + 1] = 7             # nothing behind the first -1 counts
        paths.append(keep)
    before = [(c.k.clone(), c.v.clone()) for c in caches]
    want = [(k.clone(), v.clone()) for k, v in before]
    tables = a["tables"].cpu().numpy()
    for (k, v), (k0, v0) in zip(want, before):
        for b, keep in enumerate(paths):
            for i, node in enumerate(keep):
                s, d = ctx[b] + node, ctx[b] + i
                k[tables[b, d // ps], d % ps] = k0[tables[b, s // ps], s % ps]
                v[tables[b, d // ps], d % ps] = v0[tables[b, s // ps], s % ps]
    new = ints([-9] * len(rows))
    lk.lora_kv_keep_rows(lk.KeepRowsProblem(lk.KVCaches(caches), a["tables"], a["lengths"], a["offsets"], ints(path), new))
    assert lk.lora_last_call_path() == (lk.PATH_KEEP, -(-layers // 64))
    for c, (k, v) in zip(caches, want):
        assert torch.equal(c.k, k) and torch.equal(c.v, v)
    assert new.tolist() == [c + len(p) for c, p in zip(ctx, paths)]


def test_keep_rows_refusals_on_the_device():
    rows, ctx = [5, 6, 7, 8], [40, 3, 0, 10]
    a = tree_case(rows, ctx, 2, 2, 64, 16, BF, fill=5.0)
    good = np.array([[1, 4, -1], [0, 2, 5], [-1, -1, -1], [3, 4, 7]], dtype=np.int32)
    k0, v0 = a["cache"].k.clone(), a["cache"].v.clone()
    lengths, offsets, tables = a["lengths"].clone(), a["offsets"].clone(), a["tables"].clone()

    def run(b, flag, path=good, lengths=lengths, offsets=offsets, tables=tables):
        a["cache"].k.copy_(k0)
        a["cache"].v.copy_(v0)
        new = ints([-7] * 4)
        lk.lora_kv_keep_rows(lk.KeepRowsProblem(lk.KVCaches([a["cache"]]), tables, lengths, offsets, ints(path), new))
        assert lk.lora_get_device_status() == flag
        got = new.tolist()
        assert got[b] == -7 and all(g >= 0 for i, g in enumerate(got) if i != b)
        for i in range(4):   # that sequence's pages are as they were
            pages = a["tables"][i, :-(-(rows[i] + ctx[i]) // 16)].long()
            same = torch.equal(a["cache"].k[pages], k0[pages]) and torch.equal(a["cache"].v[pages], v0[pages])
            assert same == (i == b or i == 2)

    for b, row in ((0, [4, 1, -1]), (0, [1, 1, -1]), (1, [0, 2, 6]), (3, [-2, 3, 4]), (3, [2 ** 31 - 1, -1, -1])):
        path = good.copy()
        path[b] = row
        run(b, lk.DEV_BAD_ROW, path=path)
    for b, n in ((0, 4), (1, -1), (3, 10 ** 9)):
        bad = lengths.clone()
        bad[b] = n
        run(b, lk.DEV_BAD_LENGTH, lengths=bad)
    for b, col, page in ((0, 2, 10 ** 6), (3, 0, -1)):
        bad = tables.clone()
        bad[b, col] = page
        run(b, lk.DEV_BAD_PAGE, tables=bad)


def test_keep_rows_nothing_to_keep():
    a = tree_case([3], [4], 2, 2, 64, 16, BF)
    new = ints([0])
    lk.lora_kv_keep_rows(lk.KeepRowsProblem(lk.KVCaches([a["cache"]]), a["tables"], a["lengths"], a["offsets"], ints(np.zeros((1, 0))), new))
    assert new.tolist() == [4]
    lk.lora_kv_keep_rows(lk.KeepRowsProblem(lk.KVCaches([a["cache"]]), a["tables"][:0], a["lengths"][:0], a["offsets"][:1], ints(np.zeros((0, 2)))))
    assert lk.lora_last_call_path() == (0, 0)
