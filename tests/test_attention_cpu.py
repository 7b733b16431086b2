"""Host side of the attention operators, without a GPU: the rotation's
frequency table, the bookkeeping of cache pages against a model of it, and the
refusals that are decided before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest

import adapter_sgmv_lora_gb300 as lk


@pytest.fixture(scope="module", autouse=True)
def _built():
    from adapter_sgmv_lora_gb300 import build
    build.build()


# -------------------------------------------------------------- frequencies --

def _turns_as_float(r):
    return r["turns"].astype(np.float64) / 2.0 ** 64


def _plain(D, theta):
    return theta ** (-2.0 * np.arange(D // 2) / D)


# A table entry is a double rounded a handful of times, 2^-50 relative, cut to the format's unit of 2^-64 turns.
@pytest.mark.parametrize("D,theta", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (256, 1e6)])
def test_rope_scalings(D, theta):
    f = _plain(D, theta)
    check = lambda r, want: np.testing.assert_allclose(_turns_as_float(r), want / (2 * math.pi), rtol=2.0 ** -50,
                                                            atol=2.0 ** -64)
    check(lk.lora_build_rope(D, theta), f)
    check(lk.lora_build_rope(D, theta, "linear", 4.0), f / 4)
    if D > 2:
        check(lk.lora_build_rope(D, theta, "ntk", 8.0), _plain(D, theta * 8.0 ** (D / (D - 2))))
    over = 8192 * f / (2 * math.pi)
    g = np.clip((over - 1) / 3, 0, 1)
    r = lk.lora_build_rope(D, theta, "parts", 8.0, 8192, 1.0, 4.0, attention_scale=1.5)
    check(r, g * f + (1 - g) * f / 8)
    assert r["attention_scale"] == 1.5
    if D > 2:  # fast pairs keep their frequency, the slowest is divided
        assert _turns_as_float(r)[0] == _turns_as_float(lk.lora_build_rope(D, theta))[0]


def test_rope_own_frequencies():
    f = [0.5, 2 * math.pi * 1.25, -2 * math.pi * 0.25, 0.0, -1e-300]
    r = lk.lora_build_rope(10, frequencies=f)
    np.testing.assert_allclose(_turns_as_float(r), [0.5 / (2 * math.pi), 0.25, 0.75, 0.0, 0.0], rtol=2.0 ** -50)


def test_rope_phase_is_exact_at_long_positions():
    """The wrapped integer product is the fractional turn: against exact integer arithmetic."""
    r = lk.lora_build_rope(128, 500000.0)
    for pos in (1, 131071, 2 ** 31 - 1, -5):
        wrapped = (np.int64(pos).astype(np.uint64) * r["turns"])
        assert [int(x) for x in wrapped] == [(pos * int(t)) % 2 ** 64 for t in r["turns"]]


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=258), dict(theta=0.0),
                                dict(theta=float("inf")), dict(theta=float("nan")),
                                dict(scaling="linear", factor=0.0), dict(scaling="ntk", factor=-1.0),
                                dict(rotary_dim=2, scaling="ntk", factor=2.0),
                                dict(scaling="parts", factor=2.0), dict(scaling="parts", factor=2.0,
                                                                        original_max_positions=10, low_turns=4.0),
                                dict(rotary_dim=2, frequencies=[float("nan")]),
                                dict(rotary_dim=4, frequencies=[1.0, 1.0], scaling="ntk", factor=2.0)])
def test_rope_refusals(kw):
    with pytest.raises(lk.LoraError) as e:
        lk.lora_build_rope(**{"rotary_dim": 64, **kw})
    assert e.value.status == 2


def test_rope_python_refusals():
    with pytest.raises(ValueError):
        lk.lora_build_rope(64, scaling="nonsense")
    with pytest.raises(ValueError):
        lk.lora_build_rope(64, frequencies=[1.0])
    assert lk.lib().lora_build_rope(64, 1e4, 0, 1.0, 0, 0.0, 0.0, None, None) == 1
    t = (ctypes.c_uint64 * 32)()
    assert lk.lib().lora_build_rope(64, 1e4, 9, 1.0, 0, 0.0, 0.0, None, t) == 2


# -------------------------------------------------------------------- pages --

class Model:
    """What the cache holds, seen from outside: each sequence's tokens as values, written through the rows and
    copies that Pages hands out."""

    def __init__(self, pages):
        self.p = pages
        n, ps = pages.refs.size, pages._c.page_size
        self.ps = ps
        self.cells = np.zeros((n, ps), dtype=np.int64)
        self.seqs = {}
        self.next = 1

    def append(self, s, n):
        rows, copies = self.p.append(s, n)
        for a, b in copies:
            self.cells[b] = self.cells[a]
        vals = list(range(self.next, self.next + n))
        self.next += n
        for r, v in zip(rows, vals):
            self.cells[r // self.ps, r % self.ps] = v
        self.seqs[s] = self.seqs.get(s, []) + vals

    def check(self):
        p, ps = self.p, self.ps
        refs = np.zeros_like(p.refs)
        for s in range(p.lengths.size):
            want = self.seqs.get(s, [])
            assert p.lengths[s] == len(want)
            have = -(-len(want) // ps)
            got = [self.cells[p.tables[s, j // ps], j % ps] for j in range(len(want))]
            assert got == want, s
            assert np.all(p.tables[s, have:] == -1)
            for g in p.tables[s, :have]:
                refs[g] += 1
        assert np.array_equal(refs, p.refs)
        free = sorted(p.free_pages[:p.num_free])
        assert free == [g for g in range(refs.size) if refs[g] == 0]


@pytest.mark.parametrize("ps,num_pages", [(1, 40), (3, 25), (16, 12)])
def test_pages_against_model(ps, num_pages):
    rng = np.random.default_rng(ps)
    S, M = 7, 9
    p = lk.Pages(num_pages, ps, S, M)
    m = Model(p)
    seen = set()
    for _ in range(1500):
        s, t = int(rng.integers(S)), int(rng.integers(S))
        what = rng.choice(["append", "append", "fork", "trim", "compact"])
        before = (p.tables.copy(), p.lengths.copy(), p.refs.copy(), p.free_pages.copy(), p.num_free)
        try:
            if what == "append":
                m.append(s, int(rng.integers(0, 2 * ps + 2)))
            elif what == "fork":
                n = int(rng.integers(0, p.lengths[s] + 1))
                p.fork(s, t, n)
                m.seqs[t] = m.seqs.get(s, [])[:n]
            elif what == "trim":
                n = int(rng.integers(0, p.lengths[s] + 1)) if rng.random() < 0.6 else 0
                p.trim(s, n)
                m.seqs[s] = m.seqs.get(s, [])[:n]
            else:
                src, dst = p.compact()
                assert not set(src) & set(dst) and len(set(dst)) == len(dst)
                m.cells[dst] = m.cells[src]
                used = p.refs.size - p.num_free
                assert np.all(p.refs[:used] > 0) and np.all(p.refs[used:] == 0)
            seen.add(what)
        except lk.LoraError as e:
            seen.add(e.status)
            after = (p.tables, p.lengths, p.refs, p.free_pages, p.num_free)
            assert all(np.array_equal(a, b) for a, b in zip(before, after))
        m.check()
    assert {"append", "fork", "trim", "compact", 2, 11} <= seen


def test_pages_copy_on_write_only_when_needed():
    p = lk.Pages(10, 4, 3, 5)
    assert p.append(0, 6)[1] == []
    p.fork(0, 1)
    p.fork(0, 2, 4)                          # whole pages only
    assert p.append(2, 1)[1] == []
    rows, copies = p.append(1, 1)            # its last page is shared and half full
    assert len(copies) == 1 and copies[0][0] == p.tables[0, 1] and copies[0][1] == p.tables[1, 1]
    assert rows.tolist() == [p.tables[1, 1] * 4 + 2]
    assert p.append(0, 1)[1] == []           # no longer shared
    p.fork(0, 1) if p.lengths[1] == 0 else None
    assert p.append(1, 0)[1] == []


def test_pages_refusals():
    for sizes in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0)):
        with pytest.raises(lk.LoraError) as e:
            lk.Pages(*sizes)
        assert e.value.status == 2
    p = lk.Pages(4, 4, 2, 3)
    for f in (lambda: p.append(2, 1), lambda: p.append(-1, 1), lambda: p.append(0, -1), lambda: p.append(0, 13),
              lambda: p.append(0, 2 ** 31 - 1), lambda: p.fork(0, 2), lambda: p.fork(-1, 0), lambda: p.fork(0, 1, 1),
              lambda: p.fork(0, 1, -1), lambda: p.trim(0, 1), lambda: p.trim(5, 0), lambda: p.trim(0, -1)):
        with pytest.raises(lk.LoraError) as e:
            f()
        assert e.value.status == 2
    p.append(0, 12)
    with pytest.raises(lk.LoraError) as e:
        p.append(1, 5)
    assert e.value.status == 11 and p.lengths[1] == 0
    with pytest.raises(lk.LoraError) as e:   # the child must be empty
        p.append(1, 1)
        p.fork(0, 1)
    assert e.value.status == 2
    big = lk._Pages(2 ** 20, 2 ** 12, 1, 1, 16, 16, 16, 16, 0)
    assert lk.lib().lora_pages_init(ctypes.byref(big)) == 2
    null = lk._Pages(1, 1, 1, 1, None, None, None, None, 0)
    assert lk.lib().lora_pages_init(ctypes.byref(null)) == 1


# ----------------------------------------------------------------- refusals --

def _cache(**kw):
    c = dict(dtype=lk.DTYPE_BF16, num_pages=4, page_size=16, num_kv_heads=2, head_dim=64, k=4096, v=8192,
             page_stride=16 * 128, token_stride=128, head_stride=64)
    c.update(kw)
    return lk._KVCache(**c)


def _ref(s):
    return ctypes.addressof(s)


CACHE_FAULTS = [(dict(dtype=5), 6), (dict(num_pages=0), 2), (dict(page_size=0), 2), (dict(num_kv_heads=0), 2),
                (dict(head_dim=0), 2), (dict(head_dim=257), 2), (dict(k=None), 1), (dict(v=None), 1),
                (dict(k=4097), 7), (dict(page_stride=100), 2), (dict(token_stride=64), 2), (dict(head_stride=63), 2),
                (dict(head_stride=-64), 2), (dict(page_stride=2 ** 62), 2),
                (dict(num_pages=2 ** 27, page_size=16), 2)]


@pytest.mark.parametrize("fault,code", CACHE_FAULTS)
def test_cache_refusals(fault, code):
    L = lk.lib()
    c, ok = _cache(**fault), _cache()
    h = lk._Heads(4096, 256, 64)
    a = lk._Attention(2, 4, h, h, 4096, 8, 8, 4096, 1.0, None)
    assert L.lora_paged_attention(_ref(a), _ref(c), 4096, 1 << 30, None) == code
    assert L.lora_attention_workspace_bytes(_ref(a), _ref(c)) == 0
    assert L.lora_attention_workspace_bytes(_ref(a), _ref(ok)) > 0
    one = (ctypes.c_int32 * 1)(0)
    two = (ctypes.c_int32 * 1)(1)
    assert L.lora_kv_copy_pages(_ref(c), 1, one, two, 1, None) == code
    pair = (lk._KVCache * 2)(ok, c)
    assert L.lora_kv_copy_pages(_ref(pair), 2, one, two, 1, None) == code
    assert L.lora_last_call_path(None) == 0


def test_attention_refusals():
    L = lk.lib()
    c = _cache()
    h = lk._Heads(4096, 256, 64)

    def call(cache=c, **kw):
        f = dict(num_seqs=2, num_heads=4, q=h, out=h, block_tables=4096, table_stride=8, max_pages=8, lengths=4096,
                 scale=1.0, lse=None)
        f.update(kw)
        a = lk._Attention(**f)
        return L.lora_paged_attention(_ref(a), None if cache is None else _ref(cache), None, 0, None)

    assert call() == 8                                       # all but the workspace
    assert call(cache=None) == 1
    assert L.lora_paged_attention(None, _ref(c), None, 0, None) == 1
    assert call(num_seqs=-1) == 2 and call(num_heads=0) == 2 and call(num_heads=3) == 2
    assert call(max_pages=-1) == 2 and call(table_stride=7) == 2
    assert call(q=lk._Heads(None, 256, 64)) == 1 and call(out=lk._Heads(None, 256, 64)) == 1
    assert call(lengths=None) == 1 and call(block_tables=None) == 1
    assert call(q=lk._Heads(8192, 0, 0)) == 8                # a broadcast query is fine
    assert call(out=lk._Heads(8192, 0, 64)) == 2             # a broadcast output is not
    assert call(out=lk._Heads(8192, 256, 32)) == 2
    assert call(out=lk._Heads(4096, 512, 64)) == 2           # over q with other strides
    assert call(q=lk._Heads(8192, -256, 64)) == 2
    assert call(q=lk._Heads(4097, 256, 64)) == 7 and call(lengths=4098) == 7 and call(lse=4097) == 7
    assert call(num_seqs=0) == 0                             # nothing to do


def test_rope_append_refusals():
    L = lk.lib()
    c = _cache()
    q, k = lk._Heads(4096, 512, 64), lk._Heads(65536, 512, 64)
    none = lk._Heads(None, 0, 0)

    def call(cache=c, **kw):
        f = dict(dtype=lk.DTYPE_BF16, num_tokens=3, num_heads=4, num_kv_heads=2, head_dim=64, rotary_dim=64, layout=0,
                 attention_scale=1.0, eps=1e-6, turns=4096, positions=4096, q=q, k=k, v=k, q_out=q, k_out=none,
                 q_weight=None, k_weight=None, cache_rows=4096)
        f.update(kw)
        r = lk._Rope(**f)
        return L.lora_rope_append(_ref(r), None if cache is None else _ref(cache), None)

    assert L.lora_rope_append(None, None, None) == 1
    assert call(dtype=3) == 6
    for bad in (dict(num_tokens=-1), dict(num_heads=-1), dict(num_heads=0, num_kv_heads=0), dict(head_dim=0),
                dict(head_dim=258), dict(rotary_dim=63), dict(rotary_dim=66), dict(rotary_dim=-2), dict(layout=2),
                dict(q=lk._Heads(4096, -1, 64)), dict(q_out=lk._Heads(8192, 512, 32)),
                dict(q_out=lk._Heads(4096, 256, 64)), dict(num_kv_heads=1), dict(cache=_cache(head_dim=32))):
        assert call(**bad) == 2, bad
    for bad in (dict(turns=None), dict(positions=None), dict(cache=None), dict(cache_rows=None), dict(q=none),
                dict(q_out=none), dict(k=none), dict(v=none), dict(cache=None, cache_rows=None)):
        assert call(**bad) == 1, bad
    assert call(cache=_cache(dtype=lk.DTYPE_F32)) == 6
    for bad in (dict(turns=4100), dict(positions=4098), dict(q_weight=4097), dict(cache_rows=4097),
                dict(q=lk._Heads(4097, 512, 64))):
        assert call(**bad) == 7, bad
    assert call(num_tokens=0) == 0
    assert L.lora_last_call_path(None) == 0


def test_copy_refusals():
    L = lk.lib()
    c = _cache()
    i32 = lambda *v: (ctypes.c_int32 * len(v))(*v)
    assert L.lora_kv_copy_pages(None, 1, i32(0), i32(1), 1, None) == 1
    assert L.lora_kv_copy_pages(_ref(c), 1, None, i32(1), 1, None) == 1
    assert L.lora_kv_copy_pages(_ref(c), -1, i32(0), i32(1), 1, None) == 2
    assert L.lora_kv_copy_pages(_ref(c), 1, i32(0), i32(1), -1, None) == 2
    for s, d in (((0,), (4,)), ((-1,), (0,)), ((0,), (0,)), ((0, 1), (1, 2)), ((0, 0), (2, 2))):
        assert L.lora_kv_copy_pages(_ref(c), 1, i32(*s), i32(*d), len(s), None) == 2
    big = _cache(num_pages=100)
    src, dst = list(range(30)), list(range(30, 60))
    for i, v in ((3, 29), (7, 31), (29, 100)):
        bad = dst[:]
        bad[i] = v
        if v == 31:
            bad[1] = 31
        assert L.lora_kv_copy_pages(_ref(big), 1, i32(*src), i32(*bad), 30, None) == 2
    assert L.lora_kv_copy_pages(_ref(c), 0, None, None, 3, None) == 0
    assert L.lora_kv_copy_pages(_ref(c), 1, None, None, 0, None) == 0
    two = (lk._KVCache * 2)(c, _cache(num_pages=5))
    assert L.lora_kv_copy_pages(_ref(two), 2, i32(0), i32(1), 1, None) == 2
    two = (lk._KVCache * 2)(c, _cache(dtype=lk.DTYPE_F32))
    assert L.lora_kv_copy_pages(_ref(two), 2, i32(0), i32(1), 1, None) == 6
    assert L.lora_last_call_path(None) == 0
