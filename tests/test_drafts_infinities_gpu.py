"""Infinities and rows of a wide range in the 4-bit base projection: the same on
every kernel, whatever the batch size selects."""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk
from test_drafts_gpu import BF, F32, Q4Case, _setup, _status_clean, codes_of, f64  # noqa: F401

pytestmark = pytest.mark.gpu

KERNELS = [(1, [64], BF, lk.PATH_MMA_Q4), (2, [200], BF, lk.PATH_MMA_Q4), (12, [200, 40], BF, lk.PATH_MMA_Q4),
           (7, [9900, 40], BF, lk.PATH_MMA_Q4), (16, [9900], BF, lk.PATH_MMA_Q4), (40, [264], BF, lk.PATH_MMA_Q4),
           (300, [4000, 40], BF, lk.PATH_TC_Q4), (700, [2056, 77], BF, lk.PATH_TC_Q4),
           (12, [61], F32, lk.PATH_GENERIC_Q4)]


@pytest.mark.parametrize("T,outs,dtype,path", KERNELS)
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_an_infinite_element_of_b(T, outs, dtype, path, value):
    """B[slot, o, k] infinite makes y[t, o] of the slot's rows an infinity with the sign of u[t, k] (NaN where two of
    opposite signs meet), on every kernel; everything else is as it was, bit for bit."""
    c = Q4Case(T, 512, outs, 64, 16, dtype, [T - T // 2, T // 3], seed=T)
    clean = c.run().clone()
    assert lk.lora_last_call_path()[0] & path
    cells = [(0, 3), (outs[0] - 1, 11), (sum(outs) - 1, 15)]
    for o, k in cells:
        c.b[0, o, k] = value
    c.run()
    rows = int(c.offs[1])
    want = clean.clone()
    sure = 0
    for o in {o for o, _ in cells}:
        j = 1 if o >= outs[0] else 0
        u = np.stack([f64(c.x[:rows]) @ f64(c.a)[0, j * c.R + k] for p, k in cells if p == o])
        with np.errstate(invalid="ignore"):
            y = (np.sign(u) * value).sum(0)      # two opposite ones in one sum are NaN
        # a sum of 512 products of about 1 / 16 in fp32 has the right sign down to 2^-12
        t = torch.from_numpy(np.flatnonzero((np.abs(u) > 2.0 ** -12).all(0))).cuda()
        assert torch.equal(c.y[t, o].nan_to_num(7.0, 8.0, 9.0), torch.from_numpy(y).cuda()[t].to(dtype).nan_to_num(7.0, 8.0, 9.0))
        want[:rows, o] = c.y[:rows, o]
        sure += len(t) / rows
    assert sure > 0.9
    assert torch.equal(c.y.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))


def last_row(T, outs, dtype, zeros=True):
    """A case whose last row has no adapter, its result, and the codes less their zeros."""
    c = Q4Case(T, 512, outs, 64, 16, dtype, [T // 2], seed=T, zeros=zeros)
    clean = c.run().clone()
    zero = 8.0 if c.zeros is None else np.repeat(f64(c.zeros), 64, axis=1)
    return c, clean, codes_of(c.q, 512) - zero


@pytest.mark.parametrize("T,outs,dtype,path", KERNELS)
@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_an_infinite_input(T, outs, dtype, path, value):
    """Every output of the row is an infinity with the sign of its weight, or NaN where that is zero, whatever finite
    values stand beside it; other rows are as they were, bit for bit."""
    c, clean, w = last_row(T, outs, dtype)
    c.x[T - 1, 70] = value
    c.x[T - 1, 71] = -np.sign(value) * 2.0 ** 17     # past fp16's range
    c.x[T - 1, 300] = 2.0 ** 100
    c.run()
    assert lk.lora_last_call_path()[0] & path
    with np.errstate(invalid="ignore"):
        want = torch.from_numpy(value * w[:, 70]).cuda().to(dtype)
    assert (w[:, 70] == 0).any() or sum(outs) < 100
    assert torch.equal(c.y[T - 1].nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
    assert torch.equal(c.y[:T - 1], clean[:T - 1])
    c.x[T - 1, 70] = 0
    c.x[T - 1, 9] = float("nan")
    c.run()
    assert torch.isnan(c.y[T - 1]).all() and torch.equal(c.y[:T - 1], clean[:T - 1])


@pytest.mark.parametrize("T,outs,dtype,path", KERNELS)
@pytest.mark.parametrize("large,small", [(2.0 ** 60, 1.0), (1.0, 2.0 ** -50), (2.0 ** 40, 2.0 ** -40), (2.0 ** 15, 2.0 ** -13),
                                         (2.0 ** -70, 2.0 ** -120), (2.0 ** 30, 1.0)])
def test_a_row_of_a_wide_range(T, outs, dtype, path, large, small):
    """A value far above the row's others where half the outputs have a weight of zero: there the others are all
    that is left."""
    c, clean, w = last_row(T, outs, dtype, zeros=False)
    c.q[::2, 35] = 0x88                              # inputs 70 and 71
    c.x[T - 1].mul_(small)
    c.x[T - 1, 70] = large
    c.run()
    assert lk.lora_last_call_path()[0] & path
    c.check()
    assert torch.equal(c.y[:T - 1, 1::2], clean[:T - 1, 1::2])
    c.x[T - 1] = 0                                   # nothing at all in the row
    c.run()
    assert (c.y[T - 1] == 0).all() and torch.equal(c.y[:T - 1, 1::2], clean[:T - 1, 1::2])
