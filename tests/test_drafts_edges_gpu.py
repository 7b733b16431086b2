"""The far ends of what the drafted tokens' calls take: high ranks, very many
rows or sequences, wide groups of heads, the longest trees, chains and paths."""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk
from test_drafts_gpu import (BF, E, F32, NAN, ROUND, Q4Case, _setup, _status_clean, check_tree, f64, ints,  # noqa: F401
                             randn, run_tree, tree_case)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,n,outs,group,R", [(5, 256, [64], 64, 320), (40, 128, [72, 16], 32, 1024), (300, 128, [130], 128, 257)])
def test_q4_high_ranks(dtype, T, n, outs, group, R):
    c = Q4Case(T, n, outs, group, R, dtype, [T // 2, T // 4], bias=True, ranks=True)
    c.run()
    assert lk.lora_last_call_path()[0] & lk.PATH_GENERIC_Q4
    c.check()


@pytest.mark.parametrize("T,n,outs,group,R,dtype,path", [(600000, 8, [8], 4, 4, F32, lk.PATH_GENERIC_Q4),
                                                        (70000, 96, [40], 32, 16, BF, lk.PATH_TC_Q4 | lk.PATH_MMA_Q4),
                                                        (2100000, 32, [8], 32, 8, BF, lk.PATH_GENERIC_Q4)])
def test_q4_very_many_rows(T, n, outs, group, R, dtype, path):
    c = Q4Case(T, n, outs, group, R, dtype, [T // 3, 17, T // 2])
    c.run()
    assert lk.lora_last_call_path()[0] & path
    c.check()


def test_q4_rows_and_outputs_around_the_kernels_borders():
    """Where one kernel for few rows gives way to another: each side of its rule."""
    for n, out, rows in ((4096, 12288, (3, 4, 5)), (1024, 12288, (8, 9, 16, 17)), (2048, 28672, (9, 16)), (4096, 4096, (2, 3))):
        for T in rows:
            c = Q4Case(T, n, [out], 128, 16, BF, [T // 2, T - T // 2], zeros=T % 2 == 0)
            c.run()
            assert lk.lora_last_call_path()[0] & lk.PATH_MMA_Q4
            c.check()


@pytest.mark.parametrize("dtype,hd,ps", [(BF, 64, 16), (BF, 128, 5), (F32, 32, 8)])
def test_tree_very_many_sequences(dtype, hd, ps):
    """Thousands of short sequences, a third of them without drafted tokens."""
    rows, ctx = [i % 3 for i in range(4000)], [i % 23 for i in range(4000)]
    a = tree_case(rows, ctx, 2, 1, hd, ps, dtype, seed=31)
    out, lse = run_tree(a)
    check_tree(a, out, lse, seqs=list(range(0, 4000, 97)) + [3998])
    n = sum(rows)
    assert torch.isfinite(out[:n]).all() and torch.isfinite(lse[:n]).all()
    again, _ = run_tree(a)
    assert torch.equal(out[:n], again[:n])


@pytest.mark.parametrize("dtype,H,Hk,hd", [(BF, 160, 1, 64), (BF, 384, 2, 128), (BF, 129, 1, 80), (F32, 160, 1, 32)])
def test_tree_wide_groups(dtype, H, Hk, hd):
    """More query heads to a key/value head than a chunk has rows."""
    a = tree_case([3, 1, 7], [40, 0, 300], H, Hk, hd, 16, dtype, seed=32, pad=1)
    out, lse = run_tree(a)
    check_tree(a, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_longest(dtype):
    """A tree of 1024 nodes (16 words), and chains longer than any mask."""
    a = tree_case([1024, 5], [33, 700], 2, 1, 64, 16, dtype, words=16, seed=33)
    out, lse = run_tree(a)
    check_tree(a, out, lse)
    a = tree_case([2500, 1], [10, 3], 2, 1, 64, 16, dtype, masks=None, seed=34)
    out, lse = run_tree(a)
    check_tree(a, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -1.0, 1e-30, 3.0])
def test_tree_scales(dtype, scale):
    a = tree_case([9, 20], [100, 0], 4, 2, 64, 16, dtype, seed=35)
    a["q"].mul_(0.1)
    out, lse = run_tree(a, scale=scale)
    check_tree(a, out, lse, scale=scale)


@pytest.mark.parametrize("dtype,kept", [(BF, 1024), (F32, 700)])
def test_keep_longest_path(dtype, kept):
    a = tree_case([1100, 3], [7, 50], 2, 2, 64, 16, dtype, masks=None, seed=36, fill=5.0)
    rng = np.random.default_rng(3)
    path = np.full((2, 1024), -1, dtype=np.int32)
    path[0, :kept] = np.sort(rng.choice(1100, size=kept, replace=False))
    path[1, :2] = [0, 2]
    k0, v0, tables = a["cache"].k.clone(), a["cache"].v.clone(), a["tables"].cpu().numpy()
    want_k, want_v = k0.clone(), v0.clone()
    for b, c in ((0, 7), (1, 50)):
        for i, node in enumerate(path[b][path[b] >= 0]):
            s, d = c + int(node), c + i
            for w, o in ((want_k, k0), (want_v, v0)):
                w[tables[b, d // 16], d % 16] = o[tables[b, s // 16], s % 16]
    new = ints([0, 0])
    lk.lora_kv_keep_rows(lk.KeepRowsProblem(lk.KVCaches([a["cache"]]), a["tables"], a["lengths"], a["offsets"], ints(path), new))
    assert torch.equal(a["cache"].k, want_k) and torch.equal(a["cache"].v, want_v)
    assert new.tolist() == [7 + kept, 52]
