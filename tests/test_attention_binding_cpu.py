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


class Calls:
    """Stands in for the library: keeps what a call hands over."""

    def __init__(self):
        self.got = None

    def lora_kv_copy_pages(self, ref, num_caches, src, dst, n, stream):
        self.got = (num_caches, np.frombuffer(src, np.int32).tolist(), np.frombuffer(dst, np.int32).tolist(), n)
        return 0


def test_copy_page_numbers_are_taken_as_they_are(monkeypatch):
    calls = Calls()
    monkeypatch.setattr(lk, "lib", lambda: calls)
    caches = lk.KVCaches([layer()])
    for good in ([3, 5], (3, 5), np.array([3, 5], np.int64), np.array([3, 5], np.uint8), [np.int32(3), 5]):
        lk.lora_kv_copy_pages(caches, good, np.array([7, 2 ** 31 - 1], np.int32), stream=0)
        assert calls.got == (1, [3, 5], [7, 2 ** 31 - 1], 2)
    lk.lora_kv_copy_pages(caches, [], [], stream=0)
    assert calls.got == (1, [], [], 0)
    calls.got = None
    for bad in ([2 ** 32 + 3, 5], np.array([2 ** 32 + 3, 5]), np.array([3, -2 ** 31 - 1]), np.array([3, 2 ** 31], np.uint32),
                np.array([2 ** 64 - 1, 3], np.uint64)):
        for pair in ((bad, [1, 2]), ([1, 2], bad)):
            with pytest.raises(lk.LoraError) as e:   # a page outside the caches
                lk.lora_kv_copy_pages(caches, *pair, stream=0)
            assert e.value.status == 2
    for bad in ([1.7, 5], np.array([3.0, 5.0]), [True, False], ["3", "5"], [2 ** 70, 3]):
        with pytest.raises(ValueError):
            lk.lora_kv_copy_pages(caches, bad, [1, 2], stream=0)
    assert calls.got is None


BIG = 2 ** 32


def test_pages_numbers_are_taken_as_they_are():
    """What passes 32 bits, or is no whole number, is not another sequence or another count."""
    for sizes in ((BIG + 4, 4, 2, 3), (4, BIG + 4, 2, 3), (4, 4, BIG + 2, 3), (4, 4, 2, BIG + 3)):
        with pytest.raises(lk.LoraError) as e:
            lk.Pages(*sizes)
        assert e.value.status == 2
    with pytest.raises(ValueError):
        lk.Pages(4, 4.5, 2, 3)
    p = lk.Pages(8, 4, 2, 3)
    p.append(np.int64(0), np.int32(6))
    before = p.tables.copy(), p.lengths.copy()
    for f in (lambda: p.append(BIG, 1), lambda: p.append(0, BIG + 1), lambda: p.append(1, -BIG + 2),
              lambda: p.fork(BIG, 1, 2), lambda: p.fork(0, BIG + 1), lambda: p.fork(0, 1, BIG + 2),
              lambda: p.trim(BIG), lambda: p.trim(0, BIG + 2), lambda: p.trim(-BIG)):
        with pytest.raises(lk.LoraError) as e:
            f()
        assert e.value.status == 2
    for f in (lambda: p.append(0.5, 1), lambda: p.append(0, 1.7), lambda: p.fork(0, 1, 2.5), lambda: p.trim(0, 2.5)):
        with pytest.raises(ValueError):
            f()
    assert np.array_equal(p.tables, before[0]) and np.array_equal(p.lengths, before[1])


def test_rope_numbers_are_taken_as_they_are():
    for kw in (dict(rotary_dim=BIG + 64), dict(rotary_dim=-BIG + 64),
               dict(rotary_dim=64, scaling="parts", factor=2.0, original_max_positions=BIG + 8192)):
        with pytest.raises(lk.LoraError) as e:
            lk.lora_build_rope(**kw)
        assert e.value.status == 2
    with pytest.raises(ValueError):
        lk.lora_build_rope(64.5)


def test_current_stream_without_torchs_private_calls(monkeypatch):
    """The short way to the current stream's handle is torch's own business: without it the public one serves."""
    import torch
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    assert lk._stream_handle(None) == 1003
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name)
        assert lk._stream_handle(None) == 77
    assert lk._stream_handle(5) == 5 and lk._stream_handle(types.SimpleNamespace(cuda_stream=9)) == 9


def test_attention_workspace_is_memory_of_the_call(monkeypatch):
    """A workspace of the host, of another device, or whose bytes are not all there never reaches the kernel."""
    import torch
    calls = []
    monkeypatch.setattr(lk, "lib", lambda: types.SimpleNamespace(
        lora_paged_attention=lambda problem, cache, ws, nbytes, stream: calls.append((ws, nbytes)) or 0))
    problem = types.SimpleNamespace(_ref=1, cache=types.SimpleNamespace(_ref=2), q=types.SimpleNamespace(device="cuda:0"))
    ws = lambda **kw: types.SimpleNamespace(**{**dict(is_cuda=True, device="cuda:0", is_contiguous=lambda: True,
                                                      data_ptr=lambda: 4096, nbytes=512), **kw})
    lk.lora_paged_attention(problem, ws(), stream=0)
    lk.lora_paged_attention(problem, None, stream=0)      # the library refuses it
    assert calls == [(4096, 512), (None, 0)]
    for bad in (torch.empty(128), ws(device="cuda:1"), ws(is_contiguous=lambda: False)):
        with pytest.raises(ValueError):
            lk.lora_paged_attention(problem, bad, stream=0)
    assert len(calls) == 2


def test_rope_table_holds_its_words():
    import torch
    t = lk.rope_to_device(lk.lora_build_rope(64), "cpu").turns
    assert lk.Rope(t, 64).turns is t and lk.Rope(t, 32).rotary_dim == 32
    for bad in (t.float(), t.int(), t.reshape(4, 8), t[:31], t[:1].expand(32), torch.cat([t, t])[::2]):
        with pytest.raises(ValueError):
            lk.Rope(bad, 64)


@pytest.mark.parametrize("kw", [dict(rotary_dim=64, scaling="linear", factor=1e-310),
                                dict(rotary_dim=4, scaling="ntk", factor=1e200),
                                dict(rotary_dim=4, theta=1e308, scaling="ntk", factor=8.0),
                                dict(rotary_dim=4, theta=1e-300, scaling="ntk", factor=1e-200),
                                dict(rotary_dim=2, frequencies=[1e300], scaling="linear", factor=1e-300),
                                dict(rotary_dim=2, frequencies=[1e300], scaling="parts", factor=1e-300,
                                     original_max_positions=1, low_turns=1e305, high_turns=1e306)])
def test_rope_frequencies_that_overflow_in_scaling(kw):
    """A scaled frequency that is not finite is an error and nothing is written, not a pair without rotation."""
    with pytest.raises(lk.LoraError) as e:
        lk.lora_build_rope(**kw)
    assert e.value.status == 2
    turns = np.full(2, 77, np.uint64)
    f = np.array(kw["frequencies"]) if "frequencies" in kw else None
    args = (kw["rotary_dim"], kw.get("theta", 1e4), lk.ROPE_SCALINGS[kw["scaling"]], kw["factor"],
            kw.get("original_max_positions", 0), kw.get("low_turns", 1.0), kw.get("high_turns", 4.0),
            None if f is None else f.ctypes.data, turns.ctypes.data)
    if kw["rotary_dim"] <= 4:
        assert lk.lib().lora_build_rope(*args) == 2 and turns.tolist() == [77, 77]


def test_in_place_strides_that_reach_nothing():
    """Over its input an output needs the same strides, but a row stride of one row (a head stride of one head)
    reaches nothing: torch gives such dimensions any stride."""
    import ctypes
    L = lk.lib()
    ref = ctypes.addressof
    cache = lk._KVCache(lk.DTYPE_BF16, 4, 16, 1, 64, 4096, 8192, 1024, 64, 64)

    def attend(seqs, heads, q, out):
        a = lk._Attention(seqs, heads, lk._Heads(4096, *q), lk._Heads(4096, *out), 4096, 8, 8, 4096, 1.0, None)
        return L.lora_paged_attention(ref(a), ref(cache), None, 0, None)

    assert attend(1, 4, (999, 64), (256, 64)) == 8          # on to the workspace
    assert attend(3, 1, (256, 64), (256, 999)) == 8
    assert attend(2, 4, (999, 64), (256, 64)) == 2
    assert attend(1, 4, (256, 128), (256, 64)) == 2

    def rotate(tokens, heads, q, q_out):
        h = lk._Heads(4096, *q)
        none = lk._Heads(None, 0, 0)
        r = lk._Rope(lk.DTYPE_BF16, tokens, heads, 1, 64, 64, 0, 1.0, 1e-6, 4096, 4096, h, h, none,
                     lk._Heads(4096, *q_out), none, None, None, 4096)
        return L.lora_rope_append(ref(r), ref(cache), None)

    assert rotate(1, 4, (999, 64), (256, 64)) == 1           # on to the missing v
    assert rotate(3, 1, (256, 64), (256, 999)) == 1
    assert rotate(2, 4, (999, 64), (256, 64)) == 2


def test_example_append_that_runs_out_of_pages(monkeypatch):
    """A step that does not fit changes no sequence: what was copied on write before the refusal has its contents."""
    from examples.attention_layer import AttentionLayer
    ps = 4
    L = object.__new__(AttentionLayer)
    L.device, L.caches, L.pages = "cpu", None, lk.Pages(5, ps, 4, 8)
    cells = np.zeros((5, ps), dtype=np.int64)

    def copy(caches, src, dst):
        cells[list(dst)] = cells[list(src)]

    monkeypatch.setattr(lk, "lora_kv_copy_pages", copy)
    read = lambda s: [int(cells[L.pages.tables[s, j // ps], j % ps]) for j in range(L.pages.lengths[s])]
    rows, positions = L._append([0, 2], [6, 8])              # four of the five pages
    cells.reshape(-1)[rows.numpy()] = np.arange(1, 15)
    assert positions.tolist() == list(range(6)) + list(range(8))
    L.pages.fork(0, 1)
    before = [read(s) for s in range(3)], L.pages.lengths.copy()
    with pytest.raises(lk.LoraError) as e:
        L._append([1, 0, 2], [1, 1, 1])                      # the fork's copy takes the last page
    assert e.value.status == 11
    assert np.array_equal(L.pages.lengths, before[1])
    assert [read(s) for s in range(3)] == before[0]
    L.pages.trim(2, 0)
    rows, _ = L._append([1, 0], [1, 1])
    cells.reshape(-1)[rows.numpy()] = [90, 91]
    assert read(1) == before[0][0] + [90] and read(0) == before[0][0] + [91]
