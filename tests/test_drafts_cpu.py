"""The verification of drafted tokens, without a GPU: tree masks against a walk
up the parents, and what the calls and the binding refuse."""
import ctypes
import types

import numpy as np
import pytest

import adapter_sgmv_lora_gb300 as lk


@pytest.fixture(scope="module", autouse=True)
def _built():
    from adapter_sgmv_lora_gb300 import build
    build.build()


def _ref(s):
    return ctypes.addressof(s)


# ------------------------------------------------------------------- trees --

@pytest.mark.parametrize("n,words", [(0, None), (1, None), (2, 1), (63, 1), (64, None), (65, None), (130, 3), (130, 16), (1024, 16)])
def test_build_tree(n, words):
    rng = np.random.default_rng(n)
    par = [int(rng.integers(-1, i)) for i in range(n)]
    t = lk.lora_build_tree(par, words)
    assert t["masks"].shape == (n, words or max(1, -(-n // 64))) and t["masks"].dtype == np.uint64
    for i in range(n):
        seen, j = set(), i
        while j >= 0:
            seen.add(j)
            j = par[j]
        bits = {64 * w + b for w, m in enumerate(t["masks"][i].tolist()) for b in range(64) if m >> b & 1}
        assert bits == seen and t["depths"][i] == len(seen) - 1


def test_build_tree_refusals():
    for par, words in (([0], None), ([-1, 1], None), ([-1, 2, 0], None), ([-2], None), ([-1] * 65, 1), ([-1], 0), ([-1], 17),
                       ([-1] * 1025, None), ([-1, 2 ** 40], None), ([-1], 2 ** 32 + 1)):
        with pytest.raises(lk.LoraError) as e:
            lk.lora_build_tree(par, words)
        assert e.value.status == 2
    for par in ([-1.0, 0.5], [[-1]], ["a"]):
        with pytest.raises(ValueError):
            lk.lora_build_tree(par)
    L = lk.lib()
    two = (ctypes.c_int32 * 2)(-1, 0)
    assert L.lora_build_tree(2, None, 1, None, None) == 1
    assert L.lora_build_tree(-1, two, 1, None, None) == 2
    assert L.lora_build_tree(2, two, 1, None, None) == 0
    depths = (ctypes.c_int32 * 2)(9, 9)
    assert L.lora_build_tree(2, two, 1, None, depths) == 0 and list(depths) == [0, 1]
    masks = (ctypes.c_uint64 * 2)(9, 9)
    assert L.lora_build_tree(2, two, 1, masks, None) == 0 and list(masks) == [1, 3]


# --------------------------------------------------------------- refusals --

def _cache(**kw):
    c = dict(dtype=lk.DTYPE_BF16, num_pages=4, page_size=16, num_kv_heads=2, head_dim=64, k=4096, v=8192,
             page_stride=16 * 128, token_stride=128, head_stride=64)
    c.update(kw)
    return lk._KVCache(**c)


def test_tree_attention_refusals():
    L = lk.lib()
    c = _cache()
    h = lk._Heads(4096, 256, 64)

    def call(cache=c, workspace=None, nbytes=0, **kw):
        f = dict(num_seqs=2, num_rows=5, num_heads=4, q=h, out=h, block_tables=4096, table_stride=8, max_pages=8,
                 lengths=4096, row_offsets=4096, masks=4096, mask_words=1, scale=1.0, lse=None)
        f.update(kw)
        a = lk._TreeAttention(**f)
        n = L.lora_tree_attention_workspace_bytes(_ref(a), None if cache is None else _ref(cache))
        rc = L.lora_tree_attention(_ref(a), None if cache is None else _ref(cache), workspace, nbytes, None)
        assert (n > 0) == (rc in (7, 8) and f["num_rows"] > 0 and (rc == 8 or workspace is not None))
        return rc

    assert call() == 8                                       # all but the workspace
    assert call(workspace=16, nbytes=100) == 8 and call(workspace=24, nbytes=1 << 32) == 7
    assert call(cache=None) == 1 and call(cache=_cache(dtype=7)) == 6 and call(cache=_cache(page_stride=100)) == 2
    assert L.lora_tree_attention(None, _ref(c), None, 0, None) == 1
    for bad in (dict(num_seqs=-1), dict(num_rows=-1), dict(num_heads=0), dict(num_heads=3), dict(max_pages=-1),
                dict(table_stride=7), dict(mask_words=0), dict(mask_words=17), dict(num_rows=2 ** 30),
                dict(num_seqs=2 ** 30), dict(out=lk._Heads(8192, 0, 64)), dict(out=lk._Heads(8192, 256, 32)),
                dict(out=lk._Heads(4096, 512, 64)), dict(q=lk._Heads(8192, -256, 64))):
        assert call(**bad) == 2, bad
    for bad in (dict(q=lk._Heads(None, 256, 64)), dict(out=lk._Heads(None, 256, 64)), dict(lengths=None),
                dict(block_tables=None), dict(row_offsets=None)):
        assert call(**bad) == 1, bad
    for bad in (dict(q=lk._Heads(4097, 256, 64)), dict(lengths=4098), dict(row_offsets=4098), dict(lse=4097),
                dict(masks=4100), dict(block_tables=4097)):
        assert call(**bad) == 7, bad
    assert call(masks=None, mask_words=0) == 8               # chains
    assert call(q=lk._Heads(8192, 0, 0)) == 8                # a broadcast query is fine
    assert call(num_seqs=0) == 0 and call(num_rows=0) == 0   # nothing to do
    assert L.lora_last_call_path(None) == 0


def test_keep_rows_refusals():
    L = lk.lib()
    c = _cache()

    def call(caches=(c,), n=None, **kw):
        f = dict(num_seqs=2, block_tables=4096, table_stride=8, max_pages=8, lengths=4096, row_offsets=4096,
                 path=8192, path_stride=3, max_kept=3, new_lengths=16384)
        f.update(kw)
        k = lk._Keep(**f)
        arr = (lk._KVCache * max(1, len(caches)))(*caches)
        return L.lora_kv_keep_rows(_ref(arr), len(caches) if n is None else n, _ref(k), None)

    for bad in (dict(num_seqs=-1), dict(max_pages=-1), dict(table_stride=7), dict(path_stride=2), dict(max_kept=-1),
                dict(max_kept=1025, path_stride=2000), dict(n=0), dict(caches=(c, _cache(num_pages=5))),
                dict(new_lengths=4096), dict(new_lengths=4100), dict(new_lengths=4092),
                dict(caches=(_cache(head_stride=63),))):
        assert call(**bad) == 2, bad
    for bad in (dict(lengths=None), dict(row_offsets=None), dict(block_tables=None), dict(path=None),
                dict(caches=(_cache(k=None),))):
        assert call(**bad) == 1, bad
    empty = lk._Keep()
    assert L.lora_kv_keep_rows(None, 1, _ref(empty), None) == 1
    assert L.lora_kv_keep_rows(_ref(c), 1, None, None) == 1
    assert call(caches=(c, _cache(dtype=lk.DTYPE_F32))) == 6
    for bad in (dict(path=8193), dict(lengths=4098), dict(new_lengths=16386), dict(row_offsets=4097),
                dict(block_tables=4097), dict(caches=(_cache(v=8193),))):
        assert call(**bad) == 7, bad
    assert call(num_seqs=0) == 0
    assert L.lora_last_call_path(None) == 0


def test_keep_rows_refuses_a_tensor_listed_twice():
    """Its rows would be moved twice."""
    L = lk.lib()
    k = lk._Keep(num_seqs=0, max_kept=3, path_stride=3)
    at = lambda i: _cache(k=4096 + 32 * i, v=4096 + 32 * i + 16)
    for n in (1, 2, 64, 128, 129, 700):
        layers = [at(i) for i in range(n)]
        arr = (lk._KVCache * n)(*layers)
        assert L.lora_kv_keep_rows(_ref(arr), n, _ref(k), None) == 0
        for bad in (_cache(k=4096, v=4096), _cache(k=4096 + 32 * (n - 1) + 16, v=1 << 20), _cache(k=1 << 20, v=4096)):
            arr = (lk._KVCache * (n + 1))(*layers, bad)
            assert L.lora_kv_keep_rows(_ref(arr), n + 1, _ref(k), None) == 2


def test_base_q4_refusals():
    L = lk.lib()

    def call(problem=None, routing=None, weight=None, workspace=None, nbytes=0, base=True):
        s = lk._Slice(4096, 16 * 100, 8192, 16 * 48, 48, 65536, 48, None, 0)
        p = dict(dtype=lk.DTYPE_BF16, num_tokens=5, in_dim=100, max_num_loras=2, max_lora_rank=16, x=4096,
                 x_row_stride=100, num_slices=1, slot_ranks=None)
        p.update(problem or {})
        p = lk._Problem(slices=(lk._Slice * 3)(s), **p)
        r = dict(lora_ids=4096, grouped_offsets=4096, num_groups=1, end=3, token_rows=None, host_grouped_offsets=None,
                 host_lora_ids=None)
        r.update(routing or {})
        w = dict(q=4096, q_row_stride=50, scales=4096, scale_row_stride=4, zeros=4097, zero_row_stride=4, group_size=32)
        w.update(weight or {})
        arr = (lk._Q4Weight * 3)(lk._Q4Weight(**w))
        r = lk._Routing(**r)
        return L.lora_base_q4_apply(_ref(p), _ref(r), _ref(arr) if base else None, workspace, nbytes, None)

    assert call() == 8                                       # all but the workspace
    assert call(workspace=4104, nbytes=1 << 30) == 7 and call(workspace=4096, nbytes=100) == 8
    assert call(base=False) == 1 and call(weight=dict(q=None)) == 1 and call(weight=dict(scales=None)) == 1
    for bad in (dict(q_row_stride=49), dict(scale_row_stride=3), dict(zero_row_stride=3), dict(group_size=0),
                dict(group_size=-32), dict(group_size=13)):
        assert call(weight=bad) == 2, bad
    assert call(weight=dict(zeros=None, zero_row_stride=0)) == 8
    assert call(weight=dict(group_size=2 ** 31 - 1, scale_row_stride=1, zero_row_stride=1)) == 8
    assert call(weight=dict(scales=4097)) == 7 and call(problem=dict(dtype=lk.DTYPE_F32), weight=dict(scales=4098)) == 7
    assert call(problem=dict(dtype=9)) == 6 and call(problem=dict(in_dim=0)) == 2 and call(problem=dict(x=None)) == 1
    assert call(routing=dict(end=6)) == 5 and call(routing=dict(num_groups=3)) == 10
    assert call(routing=dict(token_rows=4096)) == 2
    assert call(problem=dict(num_tokens=0), routing=dict(num_groups=0, end=0)) == 0
    assert L.lora_last_call_path(None) == 0


# ---------------------------------------------------------------- binding --

def tensor(shape, dtype, device="cuda:0", strides=None):
    """What the binding's checks look at of a CUDA tensor."""
    import torch
    t = torch.empty(shape, dtype=dtype)
    t = t if strides is None else torch.empty_strided(shape, strides, dtype=dtype)
    return types.SimpleNamespace(shape=t.shape, dtype=dtype, is_cuda=True, device=device, dim=t.dim, stride=t.stride,
                                 data_ptr=lambda: 4096, is_contiguous=t.is_contiguous, numel=t.numel)


def layer(device="cuda:0"):
    import torch
    c = object.__new__(lk.KVCache)
    t = types.SimpleNamespace(device=device, is_cuda=True, dtype=torch.bfloat16)
    for name, value in (("k", t), ("v", t), ("_struct", _cache())):
        object.__setattr__(c, name, value)
    return c


def test_tree_problem_checks():
    import torch
    BF, I32, I64 = torch.bfloat16, torch.int32, torch.int64
    good = dict(q=tensor((5, 4, 64), BF), out=tensor((5, 4, 64), BF), cache=layer(), block_tables=tensor((2, 8), I32),
                lengths=tensor((2,), I32), row_offsets=tensor((3,), I32), masks=tensor((5, 1), I64))
    p = lk.TreeAttentionProblem(**good)
    assert (p._struct.num_seqs, p._struct.num_rows, p._struct.num_heads, p._struct.mask_words) == (2, 5, 4, 1)
    assert lk.TreeAttentionProblem(**{**good, "masks": None})._struct.mask_words == 0
    for bad in (dict(q=tensor((5, 64), BF)), dict(q=tensor((5, 4, 32), BF)), dict(out=tensor((4, 4, 64), BF)),
                dict(out=tensor((5, 4, 64), torch.float32)), dict(block_tables=tensor((16,), I32)),
                dict(block_tables=tensor((2, 8), I64)), dict(lengths=tensor((3,), I32)),
                dict(row_offsets=tensor((2,), I32)), dict(masks=tensor((4, 1), I64)), dict(masks=tensor((5,), I64)),
                dict(masks=tensor((5, 1), I32)), dict(masks=tensor((5, 2), I64, strides=(1, 5))),
                dict(lse=tensor((5, 4), BF)), dict(lse=tensor((5, 3), torch.float32)),
                dict(lengths=tensor((2,), I32, "cuda:1")), dict(cache=layer("cuda:1"))):
        with pytest.raises(ValueError):
            lk.TreeAttentionProblem(**{**good, **bad})


def test_keep_problem_checks():
    import torch
    I32 = torch.int32
    good = dict(caches=lk.KVCaches([layer()]), block_tables=tensor((2, 8), I32), lengths=tensor((2,), I32),
                row_offsets=tensor((3,), I32), path=tensor((2, 4), I32), new_lengths=tensor((2,), I32))
    p = lk.KeepRowsProblem(**good)
    assert (p._struct.num_seqs, p._struct.max_kept, p._struct.path_stride) == (2, 4, 4)
    for bad in (dict(caches=lk.KVCaches([])), dict(path=tensor((3, 4), I32)), dict(path=tensor((8,), I32)),
                dict(path=tensor((2, 4), torch.int64)), dict(path=tensor((2, 4), I32, strides=(1, 2))),
                dict(new_lengths=tensor((3,), I32)), dict(lengths=tensor((2,), torch.int64)),
                dict(path=tensor((2, 4), I32, "cuda:1"))):
        with pytest.raises(ValueError):
            lk.KeepRowsProblem(**{**good, **bad})


def test_q4_weight_checks():
    import torch
    U8, BF = torch.uint8, torch.bfloat16
    q, s, z = tensor((48, 50), U8), tensor((48, 4), BF), tensor((48, 4), U8)
    assert lk.Q4Weight(q, s, np.int64(32), zeros=z).group_size == 32
    for args, kw in (((tensor((48, 50), torch.int8), s, 32), {}), ((q, tensor((47, 4), BF), 32), {}),
                     ((q, tensor((48, 4), torch.float16), 32), {}), ((q, s, 32), dict(zeros=tensor((48, 3), U8))),
                     ((q, s, 32), dict(zeros=tensor((48, 4), BF))), ((q, s, 31.5), {}),
                     ((tensor((48, 50), U8, strides=(1, 48)), s, 32), {}), ((q, tensor((48, 4), BF, "cuda:1"), 32), {})):
        with pytest.raises(ValueError):
            lk.Q4Weight(*args, **kw)
    for group in (0, -1, 2 ** 32 + 32):
        with pytest.raises(lk.LoraError) as e:
            lk.Q4Weight(q, s, group)
        assert e.value.status == 2
