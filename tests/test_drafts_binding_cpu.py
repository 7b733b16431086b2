"""What the binding hands over for a 4-bit base projection, without a GPU:
tensors are stand-ins with the attributes that it looks at."""
import ctypes
import gc
import weakref

import numpy as np
import pytest

import adapter_sgmv_lora_gb300 as lk


class Tensor:
    """What the binding looks at of a CUDA tensor; each has an address of its own."""
    addresses = iter(range(1 << 20, 1 << 30, 1 << 12))

    def __init__(self, shape, dtype, device="cuda:0"):
        import torch
        t = torch.empty(shape, dtype=dtype)
        self.at = next(self.addresses)
        self.shape, self.dtype, self.device, self.is_cuda, self.nbytes = t.shape, dtype, device, True, t.nbytes
        self.dim, self.stride, self.numel, self.element_size = t.dim, t.stride, t.numel, t.element_size
        self.is_contiguous, self.data_ptr = t.is_contiguous, lambda: self.at


class Calls:
    """Stands in for the library: keeps copies of what a call hands over."""

    def lora_base_q4_apply(self, problem, routing, base, workspace, nbytes, stream):
        take = lambda t, at: t.from_buffer_copy(ctypes.string_at(at, ctypes.sizeof(t)))
        self.problem, self.routing = take(lk._Problem, problem), take(lk._Routing, routing)
        self.base = take(lk._Q4Weight * 3, base)
        return 0


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(lk, "lib", lambda: c)
    monkeypatch.setattr(lk, "_on_current", lambda t: None)
    return c


def made(T=5, outs=(48, 16), n=96, S=2, R=16):
    import torch
    BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
    x, y = Tensor((T, n), BF), Tensor((T, sum(outs)), BF)
    a, b = Tensor((S, len(outs) * R, n), BF), Tensor((S, sum(outs), R), BF)
    problem = lk.fused_problem(x, a, b, y, outs)
    weights = [lk.Q4Weight(Tensor((o, n // 2), U8), Tensor((o, n // 32), BF), 32) for o in outs]
    offsets = np.array([0, T - 1], np.int32)
    routing = lk.Routing(Tensor((1,), I32), Tensor((2,), I32), 1, T - 1, host_grouped_offsets=offsets)
    return lk.BaseQ4Problem(problem, routing, weights), Tensor((4096,), torch.float32)


def test_fields_set_after_construction_count(calls):
    """As for the 16-bit projection, a call takes the problem, its slices and the routing as they are."""
    import torch
    BF, I32 = torch.bfloat16, torch.int32
    q4, ws = made()
    p, r = q4.problem, q4.routing
    lk.lora_base_q4_apply(q4, ws, stream=0)
    assert calls.problem.x == p.x.at and calls.problem.num_tokens == 5 and calls.routing.end == 4
    assert [calls.base[j].q for j in range(2)] == [w.q.at for w in q4.weights]
    p.x, y = Tensor((7, 96), BF), Tensor((7, 64), BF)
    for s in p.slices:
        s.y = y
    lk.lora_base_q4_apply(q4, ws, stream=0)
    assert (calls.problem.x, calls.problem.num_tokens) == (p.x.at, 7)
    assert [calls.problem.slices[j].y for j in range(2)] == [y.at, y.at + 96]
    p.slices[1].B, p.slices[1].B_offset = Tensor((2, 16, 16), BF), 0
    p.slices[0].bias, p.slices[0].bias_slot_stride = Tensor((2, 64), BF), 64
    p.slot_ranks = Tensor((2,), I32)
    r.lora_ids, r.grouped_offsets, r.end = Tensor((1,), I32), Tensor((2,), I32), 6
    r.host_grouped_offsets = np.array([0, 6], np.int32)
    lk.lora_base_q4_apply(q4, ws, stream=0)
    got = calls.problem
    assert got.slices[1].B == p.slices[1].B.at and got.slices[0].bias == p.slices[0].bias.at
    assert got.slot_ranks == p.slot_ranks.at
    assert (calls.routing.lora_ids, calls.routing.grouped_offsets) == (r.lora_ids.at, r.grouped_offsets.at)
    assert calls.routing.end == 6 and calls.routing.host_grouped_offsets == r.host_grouped_offsets.ctypes.data
    r.num_groups, r.end = 0, 0
    lk.lora_base_q4_apply(q4, ws, stream=0)
    assert (calls.routing.num_groups, calls.routing.end) == (0, 0)


def test_fields_that_do_not_fit_are_refused_by_the_call(calls):
    import torch
    q4, ws = made()
    x = q4.problem.x
    for bad in (Tensor((5, 128), torch.bfloat16), Tensor((5, 96), torch.float32), Tensor((5, 96), torch.bfloat16, "cuda:1")):
        q4.problem.x = bad
        for _ in range(2):
            with pytest.raises(ValueError):
                lk.lora_base_q4_apply(q4, ws, stream=0)
    q4.problem.x = x
    lk.lora_base_q4_apply(q4, ws, stream=0)
    assert calls.problem.x == x.at


def test_problems_that_share_a_routing_are_made_ready_once(calls):
    """The layers of a model: a problem of one does not undo another's."""
    a, ws = made()
    b = lk.BaseQ4Problem(made()[0].problem, a.routing, made()[0].weights)
    first = a._made, b._made
    for q4 in (a, b, a, b):
        lk.lora_base_q4_apply(q4, ws, stream=0)
        assert calls.problem.x == q4.problem.x.at
    assert a._made is first[0] and b._made is first[1]


def test_what_a_call_reads_lives(calls):
    """A tensor that the arguments name is held until a call has new ones."""
    import torch
    q4, ws = made()
    old = weakref.ref(q4.problem.x)
    q4.problem.x = Tensor((5, 96), torch.bfloat16)
    gc.collect()
    assert old() is not None
    lk.lora_base_q4_apply(q4, ws, stream=0)
    del calls.problem
    gc.collect()
    assert old() is None
