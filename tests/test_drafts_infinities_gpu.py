"""Infinities in the 4-bit base projection: the same on every kernel, whatever
the batch size selects."""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk
from test_drafts_gpu import BF, F32, NAN, Q4Case, _setup, _status_clean, f64  # noqa: F401

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
