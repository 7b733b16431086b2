"""What tree attention does with its probabilities: their bits, and what they
make of infinite values."""
import numpy as np
import pytest
import torch

from test_drafts_gpu import (BF, E, F32, ROUND, _setup, _status_clean, check_tree, f64, run_tree,  # noqa: F401
                             tree_case)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,H,Hk,hd,ps", [(BF, 8, 8, 32, 16), (BF, 32, 4, 64, 16), (BF, 32, 4, 128, 8),
                                              (BF, 12, 2, 128, 16), (BF, 8, 2, 256, 16), (BF, 8, 2, 128, 5),
                                              (BF, 8, 2, 256, 5), (BF, 8, 2, 33, 16), (F32, 8, 8, 64, 16)])
def test_probabilities_keep_fp32_bits(dtype, H, Hk, hd, ps):
    """Two tokens whose weighted values nearly cancel, so the output is what the probabilities' last bits leave.

    Scores are 0 and s in (-0.7, 0), one product each.  With weights w, each error times w1 |a| + w2 |b|: the exponential
    is good to 2^-22 = 4 e, the score's two roundings move it by 2 e |s| log2(e), the sum, its factor and the division are
    4 e, the terms' sum is off by 2 e; the products of 8 by 8 bits are exact, and what each of the three steps of the
    instruction cuts off is 2 e of what that step adds (1, 2^-7 and 2^-15 of the whole) and of what stands there.
    Together below 16 e, and the output's own rounding.  Terms of 16 bits are off by up to 256 e."""
    B, n = 64, 2
    rng = np.random.default_rng(hd + H)
    a = tree_case([1] * B, [n - 1] * B, H, Hk, hd, ps, dtype, masks=None, seed=21)
    kc, vc, tables = a["cache"].k, a["cache"].v, a["tables"].cpu().numpy()
    scale = 1.0 / hd ** 0.5
    q = np.zeros((B, Hk, hd))
    q[:, :, 0] = f64(torch.tensor(rng.uniform(0.3, 1.0, size=(B, Hk))).to(torch.bfloat16))
    k1 = f64(torch.tensor(-rng.uniform(0.05, 0.65, size=(B, Hk)) / scale).to(torch.bfloat16))
    p = np.exp(q[:, :, 0] * k1 * scale)
    # the pairs of 8-bit values whose ratio is nearest p, one for each column
    m = np.arange(128, 256) / 128.0
    ratio = (m[:, None] / (2 * m[None, :])).ravel()    # 1/4 .. 1
    v = np.zeros((B, n, Hk, hd))
    for b in range(B):
        for h in range(Hk):
            best = np.argsort(np.abs(ratio - p[b, h]))[:hd]
            v[b, 0, h], v[b, 1, h] = m[best // 128], -2 * m[best % 128]
    a["q"].copy_(torch.from_numpy(np.repeat(q, H // Hk, axis=1)))
    for b in range(B):
        for j in range(n):
            page, off = int(tables[b, j // ps]), j % ps
            kc[page, off] = 0
            if j == 1:
                kc[page, off, :, 0] = torch.from_numpy(k1[b]).to(kc)
            vc[page, off] = torch.from_numpy(v[b, j]).to(vc)
    out, _ = run_tree(a)
    v0, v1 = (np.repeat(v[:, j], H // Hk, axis=1) for j in (0, 1))
    pp = np.repeat(p, H // Hk, axis=1)[:, :, None]
    ref = (v0 + pp * v1) / (1 + pp)
    size = (np.abs(v0) + pp * np.abs(v1)) / (1 + pp)
    err = np.abs(f64(out) - ref)
    bound = 16 * E * size + ROUND[dtype] * np.abs(ref) * (1 + 1e-3)
    assert np.all(err <= bound), (err / size).max() / E


@pytest.mark.parametrize("dtype,H,Hk,hd,ps", [(BF, 16, 2, 128, 16), (BF, 8, 1, 64, 8), (BF, 4, 1, 256, 16),
                                              (BF, 8, 2, 128, 5), (BF, 6, 2, 200, 3), (F32, 8, 2, 64, 16)])
@pytest.mark.parametrize("ctx", [1, 50, 3000])
def test_infinite_context_values(dtype, H, Hk, hd, ps, ctx):
    """An infinite value of the context that has weight is that infinity in its column for every row, two opposite
    ones are NaN, and no other column sees them."""
    rows = [9, 2]
    a = tree_case(rows, [ctx, 17], H, Hk, hd, ps, dtype, seed=22)
    a["q"].mul_(0.3)
    tables = a["tables"].cpu().numpy()
    cells = [(ctx // 2, 3, float("inf")), (ctx - 1, 5, float("-inf"))]
    cells += [(0, 6, float("inf")), (ctx - 1, 6, float("-inf"))] if ctx > 1 else []
    for j, d, value in cells:
        a["cache"].v[int(tables[0, j // ps]), j % ps, :, d] = value
        a["v"][0][j, :, d] = 0
    out, lse = run_tree(a)
    got = out[:rows[0]].float()
    assert torch.all(torch.isposinf(got[..., 3])) and torch.all(torch.isneginf(got[..., 5]))
    if ctx > 1:
        assert torch.all(torch.isnan(got[..., 6]))
    for d in {d for _, d, _ in cells}:
        out[:rows[0], :, d] = 0
        a["v"][0][:, :, d] = 0
    check_tree(a, out, lse)


@pytest.mark.parametrize("dtype,H,Hk,hd,ps", [(BF, 16, 2, 128, 16), (BF, 8, 2, 128, 5), (BF, 8, 2, 64, 16), (BF, 4, 1, 256, 16),
                                              (BF, 4, 2, 33, 16), (F32, 8, 2, 64, 16)])
@pytest.mark.parametrize("value", [1.0, float("inf"), float("nan")])
@pytest.mark.parametrize("ctx", [0, 3, 200, 6000])
def test_scores_of_minus_infinity_alone(dtype, H, Hk, hd, ps, value, ctx):
    """A row whose every score is -inf gives 0 and lse -inf, whatever the values that have no weight."""
    rows = [5, 3]
    a = tree_case(rows, [ctx, 40], H, Hk, hd, ps, dtype, masks=None, seed=23)
    tables = a["tables"].cpu().numpy()
    a["q"].abs_().add_(0.5)
    for j in range(ctx + rows[0]):
        a["cache"].k[int(tables[0, j // ps]), j % ps, :, 0] = -float("inf")
        a["cache"].v[int(tables[0, j // ps]), j % ps, :, 1:] = value
    out, lse = run_tree(a)
    assert torch.isneginf(lse[:rows[0]]).all() and (out[:rows[0]] == 0).all()
    check_tree(a, out, lse, skip=(0,))
