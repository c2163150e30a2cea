"""A decoder layer's decode step out of the library's operators, with random weights.

Per layer: the residual's addition and the norm (``RmsNorm``), the qkv projection in 2 bits (BPDQ), the norm of every
query and key head in place, the new token into the paged cache with queries and keys turned on the way (``append``),
attention over the cache (``PagedKV``, or ``PagedKV4`` in 4 bits; with ``--blocks`` only over the blocks of 64 tokens
that promise the most to the queries), the output projection in 4 bits, the second norm straight to 8-bit activations,
the gate and up projections in 4 bits from those, and the down projection in 2 bits.  Sequences of different lengths
decode together; a step is captured once as a CUDA graph and replayed.

    python examples/decode_step.py --layers 4 --batch 8 --steps 64 --cache-bits 4
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import dequant_gemv_q2_gb300 as q2
import synth


class Layer:
    """One layer's weights and operators.  ``canonical`` keeps what the packers were given."""

    def __init__(self, hidden, q_heads, kv_heads, dim, ffn, batch, seed):
        self.Hq, self.Hk, self.D, self.ffn = q_heads, kv_heads, dim, ffn
        rng = np.random.default_rng(seed)
        gain = lambda n: (1 + 0.1 * rng.normal(size=n)).astype(np.float16)
        c = self.canonical = {
            "norm1": gain(hidden), "norm2": gain(hidden), "norm_q": gain(dim), "norm_k": gain(dim),
            "qkv": synth.bpdq((q_heads + 2 * kv_heads) * dim, hidden, seed),
            "o": synth.int4(hidden, q_heads * dim, 128, seed + 1),
            "gate_up": synth.int4(2 * ffn, hidden, 64, seed + 2, zeros=False),
            "down": synth.bpdq(hidden, ffn, seed + 3),
        }
        self.norm1, self.norm2, self.norm_q, self.norm_k = (q2.RmsNorm(c[k]) for k in ("norm1", "norm2", "norm_q", "norm_k"))
        two = lambda d: q2.Packed(q2.q2_pack_bpdq(d["plane0"], d["plane1"], d["coef"]), ntok_max=batch)
        four = lambda d: q2.Packed(q2.q2_pack_int4(d["code"], d["scale"], d["zero"], d["group"]), ntok_max=batch)
        self.qkv, self.o, self.gate_up, self.down = two(c["qkv"]), four(c["o"]), four(c["gate_up"]), two(c["down"])
        new = lambda n, t=torch.float16: torch.empty((batch, n), dtype=t, device="cuda")
        self.x, self.x8, self.s8 = new(hidden), new(hidden, torch.int8), torch.empty(batch, dtype=torch.float32, device="cuda")
        self.heads, self.att, self.gu = new((q_heads + 2 * kv_heads) * dim), new(q_heads * dim), new(2 * ffn)

    def step(self, h, delta, cache, lens, rope, blocks=None):
        """h += delta (h the residual stream, in place), then the layer; returns its last projection, not yet added."""
        D, Hq, Hk = self.D, self.Hq, self.Hk
        self.norm1.apply(delta, residual=h, out=self.x)
        self.qkv.gemv(self.x, self.heads)
        q, k, v = (t.unflatten(1, (-1, D)) for t in self.heads.split([Hq * D, Hk * D, Hk * D], dim=1))
        self.norm_q.apply(q, out=q)
        self.norm_k.apply(k, out=k)
        cache.append(k, v, lens, q=q, rope=rope)
        sel = None if blocks is None else cache.select(q, lens, blocks)
        cache.attend(q, lens, out=self.att.unflatten(1, (Hq, D)), blocks=sel)
        delta = self.o.gemv(self.att)
        self.norm2.apply(delta, residual=h, out8=self.x8, scale8=self.s8)
        self.gate_up.gemv_x8(self.x8, self.s8, self.gu)
        gate, up = self.gu.split(self.ffn, dim=1)
        return self.down.gemv(torch.nn.functional.silu(gate) * up)


class Decoder:
    """Layers, their caches and the state of a batch of sequences: page table, lengths, residual stream.

    ``bits``: of the cache, 16 or 4 (groups of 64 columns); ``blocks``: how many blocks of 64 tokens a key-value head
    attends, all if None.
    """

    def __init__(self, layers, hidden, q_heads, kv_heads, dim, ffn, batch, room, page=16, seed=0, bits=16, blocks=None):
        self.layers = [Layer(hidden, q_heads, kv_heads, dim, ffn, batch, seed + 10 * i) for i in range(layers)]
        per, g = -(-room // page), torch.Generator(device="cuda").manual_seed(seed)
        pages = torch.randperm(batch * per, device="cuda", generator=g).to(torch.int32)
        self.table, self.dim = pages.view(batch, per), dim
        pool = lambda *tail: torch.zeros((batch * per, *tail), dtype=torch.float16, device="cuda")
        kept = lambda: None if blocks is None else pool(-(-page // q2.BLOCK), kv_heads, 2, dim)
        if bits == 16:
            self.caches = [q2.PagedKV(pool(page, kv_heads, dim), pool(page, kv_heads, dim), self.table, q_heads, bounds=kept())
                           for _ in range(layers)]
        else:
            self.caches = [q2.PagedKV4.empty(batch * per, page, kv_heads, dim, 64, self.table, q_heads, bounds=blocks is not None)
                           for _ in range(layers)]
        self.blocks = blocks
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.h = torch.zeros((batch, hidden), dtype=torch.float16, device="cuda")
        self.last = torch.zeros((batch, hidden), dtype=torch.float16, device="cuda")   # what is still to be added to h
        self.rope = q2.Rope.of(dim, per * page)

    def step(self):
        """One more token per sequence: ``h`` holds its embedding on entry; afterwards ``h + last`` is the hidden state."""
        self.lens += 1
        delta = torch.zeros_like(self.h)
        for layer, cache in zip(self.layers, self.caches):
            delta = layer.step(self.h, delta, cache, self.lens, self.rope, self.blocks)
        self.last.copy_(delta)

    def capture(self):
        """The step as a graph.  Lengths, caches and the residual stream stay as they are: a step that makes what is made
        once runs before with sequences of no tokens, which stores nothing."""
        state = [(t, t.clone()) for t in (self.lens, self.h, self.last)]
        self.lens.fill_(-1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        for t, before in state:
            t.copy_(before)
        return graph


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("layers", 2), ("hidden", 4096), ("q-heads", 32), ("kv-heads", 8), ("dim", 128), ("ffn", 12288), ("batch", 4), ("steps", 64)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--cache-bits", type=int, default=16, choices=(16, 4))
    p.add_argument("--blocks", type=int, help="blocks of 64 tokens that a key-value head attends (all)")
    p.add_argument("--past", type=int, default=256, help="sequences have fewer tokens than this already (0: none)")
    a = p.parse_args()
    q2.load(build_if_missing=True)
    d = Decoder(a.layers, a.hidden, a.q_heads, a.kv_heads, a.dim, a.ffn, a.batch, room=a.steps + a.past + 44, bits=a.cache_bits, blocks=a.blocks)
    # sequences that have 0, 37, 74, .. tokens already: prompts of random keys and values
    past = torch.arange(a.batch, dtype=torch.int32, device="cuda") * 37 % max(a.past, 1)
    starts = torch.nn.functional.pad(past.cumsum(0), (1, 0)).to(torch.int32)
    rows = lambda: torch.randn(int(starts[-1]), a.kv_heads, a.dim, device="cuda").half()
    for cache in d.caches:
        cache.append(rows(), rows(), past, starts=starts, rope=d.rope)
    d.lens.copy_(past)
    graph = d.capture()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        d.h.normal_()
        graph.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    if q2.device_errors() or not torch.isfinite(d.h + d.last).all():
        raise SystemExit("the step went wrong")
    print(f"{a.layers} layers, batch {a.batch}, lengths {d.lens.tolist()}: {t * 1e6:.0f} us per step, {a.batch / t:.0f} tokens/s")


if __name__ == "__main__":
    main()
