"""What paged attention does with its probabilities: their bits and what they
make of infinite values."""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk
from test_attention_gpu import (BF, E, F32, ROUND, _setup, _status_clean, check_attention, f64,  # noqa: F401
                                make_attention, run_attention)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,H,Hk,hd,ps", [(BF, 8, 8, 32, 16), (BF, 32, 4, 64, 16), (BF, 32, 4, 128, 8),
                                              (BF, 32, 2, 128, 16), (BF, 8, 2, 256, 16), (BF, 32, 2, 256, 16),
                                              (BF, 8, 2, 128, 5), (F32, 8, 8, 64, 16)])
def test_probabilities_keep_fp32_bits(dtype, H, Hk, hd, ps):
    """Two tokens whose weighted values nearly cancel, so the output is what the probabilities' last bits leave.

    Scores are 0 and s in (-0.7, 0), one product each.  With weights w: the exponential is good to 2^-22 = 4 e, the
    score's two roundings move it by 2 e |s| log2(e), its sum and the division are 3 e; the products cancel within the
    leading bits, so their sum is exact.  Together below 12 e (w1 |a| + w2 |b|), and the output's own rounding."""
    B, n = 64, 2
    rng = np.random.default_rng(hd + H)
    a = make_attention([n] * B, H, Hk, hd, ps, dtype, "token", seed=21)
    kc, vc = a["cache"].k, a["cache"].v
    scale = 1.0 / hd ** 0.5
    q = np.zeros((B, Hk, hd))
    q[:, :, 0] = f64(torch.tensor(rng.uniform(0.3, 1.0, size=(B, Hk))).to(torch.bfloat16))
    k1 = f64(torch.tensor(-rng.uniform(0.05, 0.65, size=(B, Hk)) / scale).to(torch.bfloat16))
    s = q[:, :, 0] * k1 * scale
    p = np.exp(s)
    # the pairs of 8-bit values whose ratio is nearest p, d of them for the d columns
    m = np.arange(128, 256) / 128.0
    ratio = (m[:, None] / (2 * m[None, :])).ravel()    # a / b: 1/4 .. 1
    v = np.zeros((B, n, Hk, hd))
    for b in range(B):
        for h in range(Hk):
            best = np.argsort(np.abs(ratio - p[b, h]))[:hd]
            v[b, 0, h], v[b, 1, h] = m[best // 128], -2 * m[best % 128]
    a["q"].copy_(torch.from_numpy(np.repeat(q, H // Hk, axis=1)))
    for b in range(B):
        for j in range(n):
            page, off = int(a["tables"][b, j // ps]), j % ps
            kc[page, off] = 0
            if j == 1:
                kc[page, off, :, 0] = torch.from_numpy(k1[b]).to(kc)
            vc[page, off] = torch.from_numpy(v[b, j]).to(vc)
    out, _ = run_attention(a)
    got = f64(out)
    v0, v1 = (np.repeat(v[:, j], H // Hk, axis=1) for j in (0, 1))
    pp = np.repeat(p, H // Hk, axis=1)[:, :, None]
    ref = (v0 + pp * v1) / (1 + pp)
    size = (np.abs(v0) + pp * np.abs(v1)) / (1 + pp)
    err = np.abs(got - ref)
    bound = 12 * E * size + ROUND[dtype] * np.abs(ref) * (1 + 1e-3)
    assert np.all(err <= bound), (err / size).max() / E


@pytest.mark.parametrize("dtype,H,Hk,hd,ps", [(BF, 16, 2, 128, 16), (BF, 18, 1, 64, 8), (BF, 8, 1, 256, 16),
                                              (BF, 8, 2, 64, 5), (F32, 8, 2, 64, 16)])
@pytest.mark.parametrize("n", [1, 50, 3000])
def test_infinite_values(dtype, H, Hk, hd, ps, n):
    """An infinite value that has weight is that infinity in its column, two opposite ones are NaN, and no other
    column sees them."""
    a = make_attention([n, 17], H, Hk, hd, ps, dtype, "token", seed=22, scale_q=0.5)
    cells = [(n // 2, 3, float("inf")), (n - 1, 5, float("-inf")), (0, 6, float("inf")), (n - 1, 6, float("-inf"))]
    for j, d, value in cells:
        if n == 1 and d == 6:
            continue
        a["cache"].v[int(a["tables"][0, j // ps]), j % ps, :, d] = value
        a["v"][0][j, :, d] = 0
    out, lse = run_attention(a)
    got = out[0].float()
    assert torch.all(torch.isposinf(got[:, 3])) and torch.all(torch.isneginf(got[:, 5]))
    if n > 1:
        assert torch.all(torch.isnan(got[:, 6]))
    for d in (3, 5, 6):
        if n > 1 or d != 6:
            out[0, :, d] = 0
            a["v"][0][:, :, d] = 0
    check_attention(a, out, lse, 1.0 / hd ** 0.5)


@pytest.mark.parametrize("dtype,H,Hk,hd,ps,tile", [(BF, 8, 8, 32, 16, 32), (BF, 64, 8, 64, 16, 32),
                                                   (BF, 32, 8, 128, 16, 16), (BF, 128, 8, 128, 8, 16),
                                                   (F32, 8, 8, 64, 16, 16)])
def test_long_sums_are_rounded(dtype, H, Hk, hd, ps, tile):
    """The second half of a context has the first half's keys and the opposite values: the output is 0 but for what
    the long sum loses.  One stream to a block, four warps, so a warp adds n / 4 tile tiles of which each has its
    opposite.

    Rounded sums: half an ulp, e |o|, a tile.  |o| rises to half the weight of all and falls again, a quarter of it on
    average (4% more for the spread of the weights).  16 e for the sums within a tile and the joins.  Cut-off sums lose
    an e |o| on average in each of two steps a tile, always to the same side."""
    n, blocks = 16384, 2 * torch.cuda.get_device_properties(0).multi_processor_count
    B = blocks // Hk
    g = torch.Generator().manual_seed(7)
    k0 = torch.randn((B, n // 2, Hk), generator=g).to(dtype).cuda()
    kc = torch.zeros((B * n // ps, ps, Hk, hd), dtype=dtype, device="cuda")
    vc = torch.ones_like(kc)
    kc.view(B, 2, n // 2, Hk, hd)[..., 0] = k0[:, None]
    vc.view(B, 2, n // 2, Hk, hd)[:, 1] = -1
    q = torch.zeros((B, H, hd), dtype=dtype, device="cuda")
    q[:, :, 0] = 0.5
    out = torch.full_like(q, float("nan"))
    tables = torch.arange(B * n // ps, dtype=torch.int32, device="cuda").view(B, -1)
    prob = lk.AttentionProblem(q=q, out=out, cache=lk.KVCache(kc, vc), block_tables=tables, scale=1.0,
                               lengths=torch.full((B,), n, dtype=torch.int32, device="cuda"))
    lk.lora_paged_attention(prob, lk.new_attention_workspace(prob))
    worst = out.double().abs().max().item()
    assert worst <= (0.26 * (n / (4 * tile)) + 16) * E * (1 + 2.0 ** -8), worst / E
