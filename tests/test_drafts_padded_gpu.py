"""Padded batches in the verification of drafted tokens: sequences without any,
whose lengths nobody has set."""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk
from test_drafts_gpu import BF, F32, _setup, _status_clean, check_tree, ints, run_tree, tree_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("length", [-1, 0, 10 ** 9, -2 ** 31, 2 ** 31 - 1])
def test_sequences_without_drafts(dtype, length):
    """Both calls of a step take the same arrays: such a sequence is not looked at, and keeps its length."""
    rows, ctx = [4, 0, 9, 0, 0], [40, 7, 3, 0, 25]
    a = tree_case(rows, ctx, 2, 2, 64, 16, dtype, fill=5.0)
    want, wlse = run_tree(a)
    lengths = a["lengths"].clone()
    for b in (1, 3, 4):
        lengths[b] = length
    a["lengths"] = lengths
    out, lse = run_tree(a)
    n = sum(rows)
    assert torch.equal(out[:n], want[:n]) and torch.equal(lse[:n], wlse[:n])
    check_tree(a, out, lse)
    path = np.full((5, 3), -1, dtype=np.int32)
    path[0, :2], path[2] = [0, 3], [2, 5, 8]
    new, k0 = ints([-9] * 5), a["cache"].k.clone()
    lk.lora_kv_keep_rows(lk.KeepRowsProblem(lk.KVCaches([a["cache"]]), a["tables"], lengths, a["offsets"], ints(path), new))
    assert lk.lora_get_device_status() == 0
    assert new.tolist() == [42, length, 6, length, length]
    tables = a["tables"].cpu().numpy()
    at = lambda b, j: (int(tables[b, j // 16]), j % 16)
    for b, keep in ((0, [0, 3]), (2, [2, 5, 8])):
        for i, node in enumerate(keep):
            assert torch.equal(a["cache"].k[at(b, ctx[b] + i)], k0[at(b, ctx[b] + node)])
    # a path names a token that such a sequence does not have
    path[3, 0] = 0
    new.fill_(-9)
    lk.lora_kv_keep_rows(lk.KeepRowsProblem(lk.KVCaches([a["cache"]]), a["tables"], lengths, a["offsets"], ints(path), new))
    assert lk.lora_get_device_status() == lk.DEV_BAD_ROW
    assert new.tolist() == [42, length, 6, -9, length]
