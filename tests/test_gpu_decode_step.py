"""The operators together, as ``examples/decode_step.py`` runs them, against plain f64.

Between the operators everything is rounded to fp16 (2^-11 of each value, a
dozen of times per layer) and once to 8 bits.  The reference rounds to 8 bits
by the same rule; where a value lies so near the middle of two steps that the
roundings before decide, it takes the other one.  Were this so for every
value, it would be an error of the size of the quantization itself: a step is
1/127 of the row's maximum, at most 5 root mean squares, so 5 / 127 / sqrt(6)
= 1.6% of the projections' inputs.  So the hidden state of a step of two
layers lies within 2 x 1.6% + 24 x 2^-11 < 4.5% (root mean square).
"""
import importlib.util
import os

import numpy as np
import pytest

from oracle import bpdq as obpdq, int4 as oint4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CFG = dict(layers=2, hidden=512, q_heads=8, kv_heads=2, dim=64, ffn=768)


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_q2_gb300 as q2
    q2.load(build_if_missing=True)
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _norm(x, w):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * w.astype(np.float64)


class Plain:
    """The same layers in f64, with keys and values in lists."""

    def __init__(self, dec, keys, values):
        self.layers, self.k, self.v = [], keys, values
        for layer in dec.layers:
            c = layer.canonical
            b = lambda d: obpdq.decode_f64(d["plane0"], d["plane1"], d["coef"])
            i = lambda d: oint4.decode_f64(d["code"], d["scale"], d["zero"], d["group"])
            self.layers.append(dict(c, qkv=b(c["qkv"]), o=i(c["o"]), gate_up=i(c["gate_up"]), down=b(c["down"])))

    def step(self, h):
        hq, hk, D, F = CFG["q_heads"], CFG["kv_heads"], CFG["dim"], CFG["ffn"]
        h = h.astype(np.float64)
        freq = 10000.0 ** (-np.arange(0, D, 2) / D)
        for n, w in enumerate(self.layers):
            x = _norm(h, w["norm1"]) @ w["qkv"].T
            att = np.zeros((len(h), hq * D))
            for b in range(len(h)):
                q, k, v = np.split(x[b].reshape(-1, D), [hq, hq + hk])
                ang = len(self.k[n][b]) * freq
                turn = lambda t: np.concatenate([t[:, : D // 2] * np.cos(ang) - t[:, D // 2:] * np.sin(ang),
                                                 t[:, D // 2:] * np.cos(ang) + t[:, : D // 2] * np.sin(ang)], axis=1)
                self.k[n][b].append(turn(_norm(k, w["norm_k"])))
                self.v[n][b].append(v)
                q, K, V = turn(_norm(q, w["norm_q"])), np.array(self.k[n][b]), np.array(self.v[n][b])
                for j in range(hq):
                    s = K[:, j // (hq // hk)] @ q[j] * D ** -0.5
                    p = np.exp(s - s.max())
                    att[b, j * D: (j + 1) * D] = p @ V[:, j // (hq // hk)] / p.sum()
            h = h + att @ w["o"].T
            y = _norm(h, w["norm2"])
            step = np.abs(y).max(-1, keepdims=True) / 127
            gu = np.rint(y / step) * step @ w["gate_up"].T
            g, u = gu[:, :F], gu[:, F:]
            h = h + (g / (1 + np.exp(-g)) * u) @ w["down"].T
        return h


@pytest.mark.parametrize("batch", [1, 3, 18])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_two_layers(ex, batch, graph):
    dec = ex.Decoder(**CFG, batch=batch, room=40, page=8, seed=5)
    lens, rng = [(11 * b) % 30 for b in range(batch)], np.random.default_rng(6)
    keys, values = ([[[] for _ in range(batch)] for _ in range(2)] for _ in range(2))
    table = dec.table.cpu().numpy()
    for n, cache in enumerate(dec.caches):              # what the sequences hold already; NaN elsewhere
        pools = [np.full(tuple(cache.k.shape), np.nan, dtype=np.float16) for _ in range(2)]
        for b, m in enumerate(lens):
            for t in range(m):
                for pool, rows in zip(pools, (keys, values)):
                    row = rng.normal(size=(CFG["kv_heads"], CFG["dim"])).astype(np.float16)
                    pool[table[b, t // 8], t % 8] = row
                    rows[n][b].append(row.astype(np.float64))
        cache.k.copy_(torch.from_numpy(pools[0]))
        cache.v.copy_(torch.from_numpy(pools[1]))
    dec.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    run = dec.capture().replay if graph else dec.step
    plain = Plain(dec, keys, values)
    for _ in range(4):
        h = rng.normal(size=(batch, CFG["hidden"])).astype(np.float16)
        dec.h.copy_(torch.from_numpy(h))
        run()
        got, want = (dec.h.double() + dec.last.double()).cpu().numpy(), plain.step(h)
        rel = np.sqrt(((got - want) ** 2).mean(-1) / (want ** 2).mean(-1))
        assert (rel < 0.045).all(), rel
    assert dec.lens.cpu().tolist() == [m + 4 for m in lens]
