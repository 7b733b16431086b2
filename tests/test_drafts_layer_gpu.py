"""The attention layer example with drafted tokens against the same layer in 64
bits: prompts on several adapters, trees and chains through 4-bit and bf16
projections, rotation at the depths, tree attention, the output projection, the
accepted rows kept, then further steps on what the cache holds.

Reference and bounds are those of the layer's decode steps
(test_attention_layer_gpu.py): a drafted token is a decode step whose cache is
its context and its own branch.
"""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk
from test_attention_layer_gpu import Reference, U, bf, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as ge
    ge.build()


def dense(w):
    """A base weight's values; of a 4-bit one scale times (code - 8)."""
    if not isinstance(w, lk.Q4Weight):
        return f64(w)
    q = w.q.cpu().numpy().astype(int)
    codes = np.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)
    return (codes - 8.0) * np.repeat(f64(w.scales), w.group_size, axis=1)[:, :codes.shape[1]]


class DraftReference(Reference):
    def __init__(self, layer):
        self.L, self.k, self.v = layer, {}, {}
        self.w_qkv, self.w_o = [dense(w) for w in layer.w_qkv], dense(layer.w_o[0])
        self.fr = 500000.0 ** (-2.0 * np.arange(layer.head_dim // 2) / layer.head_dim)

    def verify(self, seq, x, parents):
        """Rows, their bounds, and each node's key and value: node j is a decode step behind its own branch."""
        k, v = self.k.get(seq, []), self.v.get(seq, [])
        nodes, rows = [], []
        for j, parent in enumerate(parents):
            branch, i = [], parent
            while i >= 0:
                branch.insert(0, i)
                i = parents[i]
            self.k[seq] = k + [nodes[i][0] for i in branch]
            self.v[seq] = v + [nodes[i][1] for i in branch]
            rows.append(self.decode(seq, x[j]))
            nodes.append((self.k[seq][-1], self.v[seq][-1]))
        self.k[seq], self.v[seq] = k, v
        return rows, nodes


def tree(rng, n):
    return [-1] + [int(rng.integers(-1, j)) for j in range(1, n)]


@pytest.mark.parametrize("group_size,page_size,heads,kv_heads,head_dim", [
    (64, 16, 8, 2, 64), (32, 8, 8, 1, 128), (None, 16, 8, 2, 64), (128, 5, 4, 4, 32)])
def test_drafts_through_the_layer(group_size, page_size, heads, kv_heads, head_dim):
    from examples.attention_layer import demo_layer
    layer = demo_layer(seed=5, group_size=group_size, page_size=page_size, num_pages=1024 // page_size,
                       max_pages=256 // page_size, heads=heads, kv_heads=kv_heads, head_dim=head_dim)
    ref = DraftReference(layer)
    rng = np.random.default_rng(2)
    draw = lambda n: torch.from_numpy(rng.standard_normal((n, layer.hidden))).to(torch.bfloat16).cuda()

    def check(got, rows, what):
        for y, (want, bound) in zip(f64(got), rows):
            err = np.abs(y - want)
            assert np.all(err <= bound), (what, (err / bound).max())

    seqs, lens = [0, 1, 2, 3], [37, 16, 1, 90]
    layer.adapter[seqs] = [1, 0, -1, 2]
    xs = [draw(n) for n in lens]
    layer.prefill(seqs, xs)
    for s, x in zip(seqs, xs):
        for row in f64(x):
            ref.store(s, row)
    layer.fork(3, 4)                              # its last page is shared
    ref.k[4], ref.v[4] = list(ref.k[3]), list(ref.v[3])
    layer.adapter[5] = 1                          # no context at all
    for step, (who, sizes) in enumerate([([0, 1, 2, 3, 4, 5], [7, 1, 66, 5, 12, 3]), ([4, 5, 0], [1, 1, 1]),
                                         ([2, 3, 1], [20, 33, 4])]):
        xs = [draw(n) for n in sizes]
        parents = [tree(rng, n) for n in sizes]
        if step == 0:
            parents[3] = [-1, 0, 1, 2, 3]         # a chain
        ys = layer.verify(who, xs, parents)
        if group_size is not None:
            assert lk.lora_last_call_path()[0] & (lk.PATH_MMA_Q4 | lk.PATH_TC_Q4)
        paths = {}
        for s, x, par, y in zip(who, xs, parents, ys):
            rows, nodes = ref.verify(s, f64(x), par)
            check(y, rows, (step, s))
            path, j = [], int(rng.integers(-1, len(par)))
            while j >= 0:
                path.insert(0, j)
                j = par[j]
            paths[s] = path
            ref.k[s] = ref.k.get(s, []) + [nodes[i][0] for i in path]
            ref.v[s] = ref.v.get(s, []) + [nodes[i][1] for i in path]
        layer.keep(paths)
        assert layer.pages.lengths[who].tolist() == [len(ref.k[s]) for s in who]
        x = draw(len(who))
        check(layer.decode(who, x), [ref.decode(s, r) for s, r in zip(who, f64(x))], (step, "decode"))
    assert lk.lora_get_device_status() == 0


def test_example_verifies_drafts(capsys):
    from examples import attention_layer
    attention_layer.verify_drafts()
    assert "verified [6, 3] drafted tokens; lengths [34, 9]" in capsys.readouterr().out
