"""The attention layer example between a verification and the word on which
drafted tokens stay: pages that move, sequences that end, other requests."""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as ge
    ge.build()


def steps(between):
    """Three requests, trees of two of them verified, `between` called, the accepted branches kept, one step on."""
    from examples.attention_layer import demo_layer
    layer = demo_layer(seed=3, group_size=64, num_pages=40, page_size=8, max_pages=20)
    g = torch.Generator().manual_seed(4)
    x = lambda n: torch.randn((n, layer.hidden), generator=g).to(layer.dtype).cuda()
    layer.adapter[[0, 1, 2]] = [1, 0, 2]
    layer.prefill([0, 1, 2], [x(30), x(21), x(11)])
    trees = [[-1, 0, 0, 1, 2, 2, 5, 6, 7], [-1, 0, 1, 1, 3]]
    layer.verify([1, 2], [x(len(t)) for t in trees], trees)
    out = between(layer, x)
    layer.keep({1: [0, 2, 5, 6], 2: [0, 1, 3, 4]})
    assert layer.pages.lengths[[1, 2]].tolist() == [25, 15]
    y = layer.decode([1, 2], x(2))
    assert lk.lora_get_device_status() == 0
    return y, out


def test_pages_that_move_before_the_branch_is_kept():
    """A request that ends and a compaction, before and after: the same rows, bit for bit."""
    def never(layer, x):
        return layer.pages.tables[[1, 2]].copy()

    def end_and_compact(layer, x):
        layer.end(0)
        assert layer.compact() > 0
        return layer.pages.tables[[1, 2]].copy()

    want, before = steps(never)
    got, after = steps(end_and_compact)
    assert not np.array_equal(before, after)
    assert torch.equal(got, want)


def test_requests_between_a_verification_and_its_end():
    def between(layer, x):
        lengths = layer.pages.lengths.copy()
        for call in (lambda: layer.decode([1], x(1)), lambda: layer.prefill([0, 2], [x(3), x(3)]),
                     lambda: layer.verify([2], [x(2)], [[-1, 0]]), lambda: layer.fork(1, 5)):
            with pytest.raises(ValueError):
                call()
            assert np.array_equal(layer.pages.lengths, lengths)
        layer.decode([0], x(1))                       # others go on
        layer.adapter[3] = 1
        layer.prefill([3], [x(9)])
        layer.verify([3], [x(3)], [[-1, 0, 0]])       # and may have drafted tokens too
        layer.fork(0, 4)

    steps(between)
    from examples.attention_layer import demo_layer
    layer = demo_layer(seed=3)
    x = lambda n: torch.randn((n, layer.hidden), device="cuda").to(layer.dtype)
    layer.keep({})                                    # nothing is there to be kept
    layer.prefill([0, 1], [x(5), x(6)])
    layer.verify([0, 1], [x(2), x(3)], [[-1, 0], [-1, 0, 0]])
    layer.end(0)
    layer.prefill([0], [x(4)])                        # a new request in its place
    layer.keep({1: [0, 2]})
    assert layer.pages.lengths[:2].tolist() == [4, 8] and lk.lora_get_device_status() == 0
