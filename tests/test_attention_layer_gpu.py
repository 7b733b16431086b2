"""The attention layer example against the same layer in 64 bits: prompts on
several adapters, forks, decode steps, an ended sequence and a compaction.

The reference rounds to bf16 where the layer does (qkv, the rotated q and k,
the attention output, y).  Where an fp32 result lies on the other side of such
a rounding an element differs by one unit, 2^-8 of it.  Bounds from that:
scores move by at most 2 * 2^-8 scale sum|q k|, the output by twice that and
2^-8 more, times the mean |v|, plus its own rounding; y by |Wo| times that.
"""
import numpy as np
import pytest
import torch

import adapter_sgmv_lora_gb300 as lk

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__ as ge
    ge.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def bf(a):
    return f64(torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16))


class Reference:
    def __init__(self, layer):
        self.L = layer
        self.k, self.v = {}, {}
        self.w_qkv, self.w_o = [f64(w) for w in layer.w_qkv], f64(layer.w_o[0])
        self.fr = 500000.0 ** (-2.0 * np.arange(layer.head_dim // 2) / layer.head_dim)

    def weights(self, slot):
        """Merged Wqkv parts and Wo of an adapter: the stacks hold bf16 values, scale folded into B."""
        L = self.L
        if slot < 0:
            return self.w_qkv, self.w_o
        R = L.a_o.shape[1]
        a, b = f64(L.a_qkv[slot]), f64(L.b_qkv[slot])
        out, off = [], 0
        for j, o in enumerate(L.qkv_dims):
            out.append(self.w_qkv[j] + b[off:off + o] @ a[j * R:(j + 1) * R])
            off += o
        return out, self.w_o + f64(L.b_o[slot]) @ f64(L.a_o[slot])

    def turn(self, x, w, pos):
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * w
        h = x.shape[-1] // 2
        c, s = np.cos(pos * self.fr), np.sin(pos * self.fr)
        return bf(np.concatenate([x[:, :h] * c - x[:, h:] * s, x[:, :h] * s + x[:, h:] * c], -1))

    def store(self, seq, x):
        L = self.L
        wq, wo = self.weights(int(L.adapter[seq]))
        pos = len(self.k.setdefault(seq, []))
        self.v.setdefault(seq, [])
        q, k, v = (bf(w @ x).reshape(-1, L.head_dim) for w in wq)
        self.k[seq].append(self.turn(k, f64(L.k_norm), pos))
        self.v[seq].append(v)
        return self.turn(q, f64(L.q_norm), pos), wo

    def decode(self, seq, x):
        L = self.L
        q, wo = self.store(seq, x)
        K, V = np.array(self.k[seq]), np.array(self.v[seq])
        o, bound = np.zeros_like(q), np.zeros_like(q)
        G, scale = L.heads // L.kv_heads, L.head_dim ** -0.5
        for h in range(L.heads):
            kk, vv = K[:, h // G], V[:, h // G]
            s = scale * kk @ q[h]
            p = np.exp(s - s.max())
            p /= p.sum()
            o[h] = p @ vv
            ds = 2 * U * scale * (np.abs(kk) @ np.abs(q[h])).max()
            bound[h] = (2 * ds + U) * (p @ np.abs(vv)) + U * np.abs(o[h])
        y = wo @ bf(o).ravel()
        return y, np.abs(wo) @ bound.ravel() + U * np.abs(y)


def test_attention_layer():
    from examples.attention_layer import demo_layer
    layer = demo_layer(seed=3, num_pages=48)
    ref = Reference(layer)
    rng = np.random.default_rng(1)
    draw = lambda n: torch.from_numpy(rng.standard_normal((n, layer.hidden))).to(torch.bfloat16).cuda()
    steps = 0

    def decode(seqs):
        nonlocal steps
        x = draw(len(seqs))
        y = f64(layer.decode(seqs, x))
        for i, s in enumerate(seqs):
            want, bound = ref.decode(s, f64(x[i]))
            err = np.abs(y[i] - want)
            assert np.all(err <= bound), (steps, s, (err / bound).max())
        steps += 1

    seqs, lens = [0, 1, 2, 3], [37, 16, 1, 90]
    layer.adapter[seqs] = [1, 0, -1, 2]
    xs = [draw(n) for n in lens]
    layer.prefill(seqs, xs)
    for s, x in zip(seqs, xs):
        for row in f64(x):
            ref.store(s, row)
    layer.fork(0, 4)
    layer.fork(3, 5)
    for child, parent in ((4, 0), (5, 3)):
        ref.k[child], ref.v[child] = list(ref.k[parent]), list(ref.v[parent])
    decode([0, 1, 2, 3, 4, 5])
    decode([5, 0, 2])
    layer.end(1)
    layer.end(3)
    for s in (1, 3):
        ref.k.pop(s), ref.v.pop(s)
    assert layer.compact() > 0
    decode([0, 2, 4, 5])
    layer.adapter[1] = 0
    decode([1, 4])                                # a new sequence, first token
    assert lk.lora_get_device_status() == 0


def test_example_runs(capsys):
    from examples import attention_layer
    attention_layer.main()
    assert "decoded (4, 256) rows" in capsys.readouterr().out
