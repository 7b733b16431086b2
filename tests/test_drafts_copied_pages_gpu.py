"""Tree attention over bf16 pages that are no whole eights of tokens, whose rows
the tensor-core kernel copies one by one, with checks and a search for
non-finite values of its own: what test_drafts_gpu.py asks of pages that come in
boxes."""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk
from test_drafts_gpu import (BF, NAN, RAGGED, _setup, _status_clean, check_tree, ints, randn, run_tree,  # noqa: F401
                             tree_case)

pytestmark = pytest.mark.gpu


def on_tc():
    return bool(lk.lora_last_call_path()[0] & lk.PATH_TC_TREE)


@pytest.mark.parametrize("masks", ["tree", "random", None])
@pytest.mark.parametrize("H,Hk,hd,ps,order", [
    (8, 2, 256, 3, "token"), (6, 2, 200, 5, "head"), (12, 4, 256, 12, "side"), (4, 4, 136, 1, "token"),
    (8, 2, 128, 5, "head"), (16, 1, 64, 7, "token"), (14, 2, 64, 20, "side"), (6, 3, 96, 12, "token"), (4, 2, 8, 9, "token")])
def test_ragged_trees(H, Hk, hd, ps, order, masks):
    rows, ctx = RAGGED
    a = tree_case(list(rows), list(ctx), H, Hk, hd, ps, BF, order, masks, pad=3, words=2 if masks == "random" else None)
    out, lse = run_tree(a)
    assert on_tc()
    check_tree(a, out, lse)
    again, lse2 = run_tree(a)
    n = sum(rows)
    assert torch.equal(out[:n], again[:n]) and torch.equal(lse[:n], lse2[:n])


@pytest.mark.parametrize("rows,ctx,hd,ps", [([60], [9000], 128, 12), ([60, 5], [7000, 3], 64, 9), ([33], [5000], 256, 12),
                                            ([200, 3], [300, 2000], 128, 5), ([13, 26, 5, 9] * 8, [700, 1500, 128, 2048] * 8, 128, 12),
                                            ([4] * 150, [30 + i for i in range(150)], 64, 5)])
def test_long_contexts_and_many_sequences(rows, ctx, hd, ps):
    """Every stage used many times over, tiles of several sequences on their way at once."""
    a = tree_case(rows, ctx, 8, 2, hd, ps, BF, seed=2)
    out, lse = run_tree(a)
    assert on_tc()
    check_tree(a, out, lse, seqs=None if len(rows) < 30 else list(range(0, len(rows), 13)) + [len(rows) - 1])


@pytest.mark.parametrize("hd,ps", [(128, 5), (64, 3), (256, 5), (200, 12), (128, 16)])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), NAN, 3e38])
def test_unseen_values_have_no_part(hd, ps, value):
    """Values of one drafted token, keys and values of another, that are infinite, NaN or huge: rows that see neither
    are the same bit for bit, a row that sees the first alone has it."""
    rows, ctx = [40, 9, 3, 70], [100, 0, 500, 250]
    a = tree_case(rows, ctx, 4, 2, hd, ps, BF, seed=4)
    clean, _ = run_tree(a)
    assert on_tc()
    kc, vc = a["cache"].k, a["cache"].v
    tables = a["tables"].cpu().numpy()
    at = 0
    for b, (n, c) in enumerate(zip(rows, ctx)):
        tok, kept = n - 2, []
        for t, both in ((tok, False), (n - 1, True)):
            page, off = int(tables[b, (c + t) // ps]), (c + t) % ps
            kept.append((page, off, kc[page, off].clone(), vc[page, off].clone()))
            vc[page, off] = value
            if both:
                kc[page, off] = value
        out, _ = run_tree(a)
        sees = a["sees"][b]
        blind = [i for i in range(n) if not sees[i, c + tok] and not sees[i, c + n - 1]]
        assert blind and torch.equal(out[at:at + n][blind], clean[at:at + n][blind])
        one = [i for i in range(n) if sees[i, c + tok] and not sees[i, c + n - 1]]
        if not np.isfinite(value):
            got = out[at:at + n][one]
            assert one and (torch.isnan(got).all() if value != value else (got == value).all())
        others = [i for i in range(sum(rows)) if not at <= i < at + n]
        assert torch.equal(out[others], clean[others])
        for page, off, k0, v0 in kept:
            kc[page, off], vc[page, off] = k0, v0
        at += n


@pytest.mark.parametrize("hd,ps", [(64, 5), (128, 12), (256, 3)])
def test_bad_lengths_pages_offsets(hd, ps):
    rows, ctx = [4, 70, 9, 3], [100, 30, 0, 700]
    a = tree_case(rows, ctx, 8, 2, hd, ps, BF, words=2)
    first = np.cumsum([0] + rows)
    lengths, tables, offsets = a["lengths"].clone(), a["tables"].clone(), a["offsets"].clone()

    def others_same(bad, flag):
        out, lse = run_tree(a)
        assert on_tc() and lk.lora_get_device_status() == flag
        for b in bad:
            assert torch.isnan(out[first[b]:first[b + 1]]).all() and torch.isnan(lse[first[b]:first[b + 1]]).all()
        check_tree(a, out, lse, skip=bad)

    for b, length in ((0, 3), (1, -5), (3, 10 ** 9), (2, 0), (2, -2 ** 31)):
        a["lengths"] = lengths.clone()
        a["lengths"][b] = length
        others_same([b], lk.DEV_BAD_LENGTH)
    a["lengths"] = lengths
    for b, token, page in ((0, 40, -1), (3, 702, 10 ** 6), (3, 0, 2 ** 31 - 1), (1, 99, -2 ** 31), (2, 0, -1)):
        a["tables"] = tables.clone()
        a["tables"][b, token // ps] = page
        others_same([b], lk.DEV_BAD_PAGE)
    a["tables"] = tables
    for i, v in ((0, -1), (2, 3), (4, 10 ** 6)):
        a["offsets"] = offsets.clone()
        a["offsets"][i] = v
        out, lse = run_tree(a)
        assert lk.lora_get_device_status() == lk.DEV_BAD_OFFSETS
        assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_in_place():
    for hd in (128, 64):
        H, Hk = 8, 2
        a = tree_case([9, 30, 2], [300, 64, 0], H, Hk, hd, 5, BF, seed=5)
        y = randn((a["N"], (H + 2 * Hk) * hd), BF, 6)
        keep, q = y.clone(), y[:, :H * hd].unflatten(1, (H, hd))
        a["q"] = q.clone()
        out, lse = run_tree(a, q=q, out=q)
        assert on_tc()
        check_tree(a, out, lse)
        assert torch.equal(y[:, H * hd:], keep[:, H * hd:])


@pytest.mark.parametrize("ps", [12, 16])
def test_far_offsets(ps):
    """Pages whose elements lie past 2^31 and 2^32 elements of the cache's start, rows on 16-byte boundaries: copied
    ones, and such as come in boxes."""
    Hk, hd, stride = 8, 128, 2 ** 31 // 3 // 16 * 16 + 16
    base = torch.empty(8 * stride, dtype=BF, device="cuda")
    kc = base.as_strided((7, ps, Hk, hd), (stride, Hk * hd, hd, 1))
    vc = base[ps * Hk * hd:].as_strided((7, ps, Hk, hd), (stride, Hk * hd, hd, 1))
    a = tree_case([5], [7 * ps - 5], 8, Hk, hd, ps, BF, seed=8)
    order = [6, 0, 5, 1, 4, 2, 3]
    for i, page in enumerate(order):
        kc[page] = a["k"][0][ps * i:ps * i + ps]
        vc[page] = a["v"][0][ps * i:ps * i + ps]
    a["cache"], a["tables"] = lk.KVCache(kc, vc), ints([order])
    out, lse = run_tree(a)
    assert on_tc()
    check_tree(a, out, lse)
