"""What the binding's objects of the attention operators check, without a GPU:
caches are stand-ins with the attributes that the checks look at."""
import types

import numpy as np
import pytest

import adapter_sgmv_lora_gb300 as lk


@pytest.fixture(scope="module", autouse=True)
def _built():
    from adapter_sgmv_lora_gb300 import build
    build.build()


def layer(device="cuda:0", num_pages=40):
    c = object.__new__(lk.KVCache)
    t = types.SimpleNamespace(device=device, is_cuda=True)
    for name, value in (("k", t), ("v", t), ("_struct", lk._KVCache(lk.DTYPE_BF16, num_pages, 16, 2, 64, 4096, 8192,
                                                                    2048, 128, 64))):
        object.__setattr__(c, name, value)
    return c


def test_caches_on_one_device():
    lk.KVCaches([layer(), layer()])
    with pytest.raises(ValueError):
        lk.KVCaches([layer(), layer(), layer("cuda:1")])


def test_caches_keep_their_layers():
    """A list that grows later does not change what was described: the count handed over is of the same layers."""
    layers = [layer()]
    caches = lk.KVCaches(layers)
    layers.append(layer())
    assert len(caches.layers) == 1 and len(caches._struct) == 1
    assert len(lk.KVCaches([]).layers) == 0
