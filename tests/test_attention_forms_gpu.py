"""The forms that a call's size picks: block tables wider than any sequence
(what a server holds), calls of many long streams with every row compared,
the rotation of many tokens, and calls inside a captured graph."""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk
from test_attention_gpu import (BF, F32, _setup, _status_clean, check_attention, make_attention,  # noqa: F401
                                pool, randn, run_attention)
from test_attention_gpu import test_rope_append as check_rope_append

pytestmark = pytest.mark.gpu


def sm_count():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------ wide tables --

@pytest.mark.parametrize("large", [True, False])
@pytest.mark.parametrize("dtype,lens,H,Hk,hd,ps,order", [
    # a warp a stream: short and many, one or two tiles and more than SMs
    (BF, [64] * 290 + [0, 1, 63, 33, 16, 0], 16, 8, 128, 16, "token"),
    (BF, [1 + 7 * i % 32 for i in range(90)], 32, 4, 128, 16, "head"),
    (F32, [1 + 5 * i % 16 for i in range(90)], 12, 4, 64, 16, "token"),
    # a block a stream
    (BF, [1 + 11 * i % 60 for i in range(30)], 16, 8, 128, 16, "token"),
    (BF, [0] + [1 + 17 * i % 100 for i in range(19)], 20, 4, 64, 8, "head"),
    (F32, [1 + 13 * i % 60 for i in range(28)], 8, 8, 64, 16, "token"),
    (BF, [1 + 13 * i % 60 for i in range(20)], 18, 2, 256, 16, "token"),
    # even pieces: all alike, and one context that outweighs the others
    (BF, [900 + 37 * i % 200 for i in range(40)], 16, 8, 128, 16, "token"),
    (BF, [200] * 17 + [40000] + [7, 0, 190] * 7, 16, 8, 128, 16, "token"),
    (BF, [50000] + [30] * 60, 16, 1, 64, 16, "head"),
    (BF, [20] * 30 + [30000, 11, 0, 100], 32, 2, 256, 16, "token"),
    (F32, [100] * 25 + [20000] + [3, 0, 150] * 5, 8, 2, 64, 16, "token"),
    (BF, [100] * 25 + [9000] + [3, 0, 150] * 5, 8, 2, 128, 1, "token"),
])
def test_tables_wider_than_sequences(dtype, lens, H, Hk, hd, ps, order, large):
    """What the table allows decides how many blocks there are and how they are joined, the lengths how the work is
    cut: the results are those of a table that fits, whatever it allows."""
    need = max(1, -(-max(lens) // ps))
    pages = 4 * need
    if large:     # 192 places a block at least, by the narrowest count of streams and the widest tile
        blocks = 2 * sm_count()
        pages = max(need, -(-192 * blocks * 32 // (len(lens) * Hk * ps)) + 1)
    a = make_attention(lens, H, Hk, hd, ps, dtype, order, seed=31, max_pages=pages)
    out, lse = run_attention(a)
    check_attention(a, out, lse, 1.0 / hd ** 0.5)
    again, lse2 = run_attention(a)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


# ---------------------------------------------------------- every row of them

def shuffled(lens, seed):
    return [lens[i] for i in np.random.default_rng(seed).permutation(len(lens))]


@pytest.mark.parametrize("dtype,lens,H,Hk,hd,order", [
    (BF, [4000, 6500, 9000, 1, 0, 5555] * 8, 16, 8, 128, "token"),
    (BF, [17000, 33, 9111, 20001, 7] * 10, 16, 4, 64, "head"),
    (F32, [2100, 7, 3333, 1500, 0, 1] * 16, 8, 8, 64, "token"),
    (BF, [1000 + 7 * i for i in range(260)] + [1, 0, 33] * 8, 4, 2, 128, "token"),
    (BF, [700, 3, 0, 1, 2500, 16] * 12, 18, 2, 256, "head"),
    # more streams than blocks, all of them
    (BF, [40] * 300, 8, 8, 64, "token"),
    (BF, [1] * 700, 4, 4, 64, "token"),
    (F32, [5] * 400, 4, 4, 64, "token"),
    (BF, [5 + 53 * i % 400 for i in range(200)], 16, 8, 64, "token"),
])
def test_every_row(dtype, lens, H, Hk, hd, order):
    """Whole streams between shared ones, in no order: every sequence against the reference."""
    lens = shuffled(lens, 5)
    a = make_attention(lens, H, Hk, hd, 16, dtype, order, seed=32)
    out, lse = run_attention(a)
    check_attention(a, out, lse, 1.0 / hd ** 0.5)


# --------------------------------------------------- rotation of many tokens

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", [
    # dtype, T, H, Hk, hd, rot, interleaved, norm, order, page_size, fused, attention scale
    (BF, 1500, 32, 8, 128, 128, False, False, "token", 16, True, 1.0),
    (BF, 1100, 32, 8, 128, 128, False, True, "head", 16, True, 1.25),
    (BF, 1301, 64, 8, 128, 64, False, False, "token", 8, True, 1.0),
    (BF, 2500, 7, 3, 128, 128, True, True, "side", 16, True, 1.1),
    (BF, 3001, 5, 1, 64, 32, True, False, "token", 24, True, 1.0),
    (BF, 2800, 6, 2, 80, 64, False, True, "head", 16, True, 1.0),
    (BF, 701, 16, 4, 256, 256, False, True, "token", 16, True, 1.0),
    (F32, 701, 32, 8, 128, 128, False, True, "token", 16, True, 1.0),
    (F32, 1777, 16, 16, 80, 32, True, False, "head", 24, True, 1.1),
    (F32, 1200, 9, 3, 256, 64, False, False, "side", 5, True, 1.0),
    # not whole 16-byte partners: element by element
    (BF, 1300, 32, 8, 80, 20, False, True, "token", 16, True, 1.0),
    (BF, 1100, 16, 2, 96, 24, False, False, "head", 16, True, 1.1),
], ids=lambda c: "-".join(str(x) for x in c[:10]).replace("torch.", ""))
def test_rope_append_many_tokens(case, in_place):
    """Above 32 groups of heads an SM a warp takes several of them in turn, the next ones loaded meanwhile."""
    dtype, T, H, Hk, hd = case[:5]
    lanes = 1
    while 2 * lanes < hd * (2 if dtype == BF else 4) // 16:
        lanes *= 2
    groups = -(-H // (32 // lanes)) + 2 * -(-Hk // (32 // lanes))
    assert T * groups > 32 * sm_count()
    check_rope_append(case, in_place)


# ------------------------------------------------------------------- graphs --

@pytest.mark.parametrize("dtype", [BF, F32])
def test_calls_in_a_captured_graph(dtype):
    """One step captured once, replayed on other positions, lengths, rows, tables and values."""
    H, Hk, hd, ps, B = 8, 2, 64, 16, 6
    first = make_attention([40, 700, 1, 0, 16, 333], H, Hk, hd, ps, dtype, "token", seed=41, spare=12, max_pages=60)
    second = make_attention([600, 17, 64, 5, 0, 90], H, Hk, hd, ps, dtype, "token", seed=42, spare=3, max_pages=60)
    pages = max(first["cache"].k.shape[0], second["cache"].k.shape[0])
    kc, vc = pool(pages, ps, Hk, hd, dtype, "token", fill=0.0)
    cache = lk.KVCache(kc, vc)
    rope = lk.rope_to_device(lk.lora_build_rope(hd))
    y = torch.zeros((B, (H + 2 * Hk) * hd), dtype=dtype, device="cuda")
    q, k, v = (t.unflatten(1, (-1, hd)) for t in y.split([H * hd, Hk * hd, Hk * hd], 1))
    positions, rows, lengths = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    tables = torch.zeros((B, 60), dtype=torch.int32, device="cuda")
    out = torch.zeros((B, H, hd), dtype=dtype, device="cuda")
    rot = lk.RopeProblem(q=q, k=k, v=v, q_out=q, rope=rope, positions=positions, cache=cache, cache_rows=rows)
    att = lk.AttentionProblem(q=q, out=out, cache=cache, block_tables=tables, lengths=lengths)
    ws, caches = lk.new_attention_workspace(att), lk.KVCaches([cache])

    def step():
        lk.lora_rope_append(rot)
        lk.lora_paged_attention(att, ws)
        lk.lora_kv_copy_pages(caches, [0], [pages - 1])

    def fill(a, seed):
        n = a["cache"].k.shape[0]
        kc.zero_(), vc.zero_()
        kc[:n] = torch.nan_to_num(a["cache"].k)
        vc[:n] = torch.nan_to_num(a["cache"].v)
        y.copy_(randn(tuple(y.shape), dtype, seed))
        tables.copy_(a["tables"])
        lens = a["lens"]
        lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        positions.copy_(torch.tensor([max(n - 1, 0) for n in lens], dtype=torch.int32))
        rows.copy_(torch.tensor([int(a["tables"][b, (n - 1) // ps]) * ps + (n - 1) % ps if n else -1
                                 for b, n in enumerate(lens)], dtype=torch.int32))

    want = []
    for a, seed in ((first, 1), (second, 2)):
        fill(a, seed)
        step()
        want.append([t.clone() for t in (out, q, kc, vc)])
    fill(first, 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 0, 1):
        fill((first, second)[i], i + 1)
        out.fill_(float("nan"))
        ws.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((out, q, kc, vc), want[i]):
            assert torch.equal(got, ref)
