"""The decode step's operators around the packed matrix-vector products, as cases that can be timed and checked.

``norm``    root-mean-square norm over rows, with the residual's addition and an fp16 and/or an 8-bit output.
``int4``    y = W x for weights of 4 bits with group scales, 1..64 tokens, x in fp16 or in 8 bits with a scale per token.
``attend``  attention of one new token per sequence over a paged key-value cache, which may take the new key and value in.

Each has a plain form (elementary operations in 32 bits, rounded once at the end), the library's form (``own``), and
its definition in 64 bits (``exact``).  Weights and hidden sizes are those of the Qwen3-8B- and 14B-shaped stacks.
"""
import math

import torch

own = False
EPS = 1e-6


def listed():
    return [
        # hidden state of one decoded token (8B width) on its way into a projection
        {"name": "norm 1x4096 residual", "op": "norm", "tokens": 1, "heads": 1, "width": 4096, "gap": 0, "residual": True, "out": "fp16"},
        # 64 tokens at the 14B width, handed to a product with 8-bit activations
        {"name": "norm 64x5120 residual int8", "op": "norm", "tokens": 64, "heads": 1, "width": 5120, "gap": 0, "residual": True, "out": "int8"},
        # the norm of every query head, read in place out of the 14B qkv projection's 7168 outputs
        {"name": "norm 64x40x128 strided", "op": "norm", "tokens": 64, "heads": 40, "width": 128, "gap": 2048, "residual": False, "out": "fp16"},
        # a long prompt's hidden states, both outputs
        {"name": "norm 16384x4096 residual both", "op": "norm", "tokens": 16384, "heads": 1, "width": 4096, "gap": 0, "residual": True, "out": "both"},
        # the 8B output projection at one token: latency counts
        {"name": "int4 4096x4096 1 token", "op": "int4", "rows": 4096, "cols": 4096, "tokens": 1, "group": 128, "zeros": False, "x": "fp16"},
        # the 8B gate and up projections at one token, weights with zero points
        {"name": "int4 24576x4096 1 token zeros", "op": "int4", "rows": 24576, "cols": 4096, "tokens": 1, "group": 128, "zeros": True, "x": "fp16"},
        # the 14B down projection for a handful of sequences, activations in 8 bits
        {"name": "int4 5120x17408 7 tokens x8", "op": "int4", "rows": 5120, "cols": 17408, "tokens": 7, "group": 64, "zeros": False, "x": "int8"},
        # the 14B gate and up projections at the largest token count
        {"name": "int4 34816x5120 64 tokens zeros", "op": "int4", "rows": 34816, "cols": 5120, "tokens": 64, "group": 128, "zeros": True, "x": "fp16"},
        # one sequence early in its answer, 8B heads: latency counts
        {"name": "attend 1x777", "op": "attend", "batch": 1, "length": 777, "ragged": False, "kv_heads": 8, "group": 4, "dim": 128, "page": 16, "order": "token", "append": True},
        # sequences of every length up to 4096 decoded together, 14B heads
        {"name": "attend 16 ragged 4096", "op": "attend", "batch": 16, "length": 4096, "ragged": True, "kv_heads": 8, "group": 5, "dim": 128, "page": 16, "order": "token", "append": True},
        # a full batch of long sequences, 8B heads, pages stored head by head
        {"name": "attend 64x8192", "op": "attend", "batch": 64, "length": 8192, "ragged": False, "kv_heads": 8, "group": 4, "dim": 128, "page": 64, "order": "head", "append": False},
        # one very long sequence: the work has to be split over its length
        {"name": "attend 1x131072", "op": "attend", "batch": 1, "length": 131072, "ragged": False, "kv_heads": 8, "group": 4, "dim": 128, "page": 256, "order": "token", "append": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "int4", "attend"])
    if op == "norm":
        heads = rng.choice([1, 1, 1, rng.randint(2, 40)])
        width = rng.choice([_log(rng, 64, 17408), 8 * _log(rng, 8, 2176)]) if heads == 1 else rng.choice([64, 96, 128, 256])
        tokens = _log(rng, 1, max(1, min(16384, (16384 * 4096) // (width * heads))))
        return {"op": "norm", "tokens": tokens, "heads": heads, "width": width, "gap": rng.choice([0, 0, 64, 2048, 5]),
                "residual": heads == 1 and rng.random() < 0.7, "out": rng.choice(["fp16", "int8", "both"])}
    if op == "int4":
        group = rng.choice([32, 64, 128])
        cols = group * _log(rng, 2, 17408 // group)
        rows = _log(rng, 16, min(34816, 34816 * 5120 // cols))
        return {"op": "int4", "rows": rows, "cols": cols, "tokens": _log(rng, 1, 64), "group": group, "zeros": rng.random() < 0.5, "x": rng.choice(["fp16", "int8"])}
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    batch = _log(rng, 1, 64)
    length = _log(rng, 1, min(131072, 64 * 8192 * 8 * 128 // (batch * kv_heads * dim)))
    return {"op": "attend", "batch": batch, "length": length, "ragged": rng.random() < 0.5, "kv_heads": kv_heads, "group": rng.choice([1, 2, 3, 4, 5, 6, 8, 16]),
            "dim": dim, "page": rng.choice([8, 16, 24, 32, 64, 100, 256]), "order": rng.choice(["token", "head"]), "append": rng.random() < 0.5}


def _lens(case):
    """The sequences' lengths: all `length`, or spread from 1 to `length`."""
    b, n = case["batch"], case["length"]
    if not case["ragged"]:
        return [n] * b
    return [n] if b == 1 else [1 + (n - 1) * ((i * 29 + b - 1) % b) // (b - 1) for i in range(b)]


def work(case):
    if case["op"] == "norm":
        rows, w = case["tokens"] * case["heads"], case["width"]
        each = 2 + (4 if case["residual"] else 0) + {"fp16": 2, "int8": 1, "both": 3}[case["out"]]
        return {"bytes": rows * w * each + 2 * w + (0 if case["out"] == "fp16" else 4 * rows), "flops": 5 * rows * w}
    if case["op"] == "int4":
        r, c, n = case["rows"], case["cols"], case["tokens"]
        groups = r * c // case["group"]
        xbytes = n * c * 2 if case["x"] == "fp16" else n * (c + 4)
        return {"bytes": r * c // 2 + 2 * groups + (groups // 2 if case["zeros"] else 0) + xbytes + 2 * n * r, "flops": 2 * r * c * n}
    tokens, kv = sum(_lens(case)), case["kv_heads"] * case["dim"]
    q = case["batch"] * kv * case["group"]
    pages = sum(-(-n // case["page"]) for n in _lens(case))
    # the new token's key and value are read once from the projection and written to the cache, instead of read from it
    return {"bytes": tokens * kv * 4 + 4 * q + 4 * pages + (4 * case["batch"] * kv if case["append"] else 0), "flops": 4 * tokens * kv * case["group"]}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if own:
        import dequant_gemv_q2_gb300 as q2
        q2.load()
    if case["op"] == "norm":
        t, h, w = case["tokens"], case["heads"], case["width"]
        s["wide"] = torch.randn(t, h * w + case["gap"], device="cuda", generator=g).half()
        # a few columns far larger than the rest, as hidden states have
        big = torch.rand(h * w + case["gap"], device="cuda", generator=g) < 0.003
        s["wide"][:, big] *= 20
        s["x"] = s["wide"][:, : h * w].unflatten(1, (h, w))
        s["weight"] = (1 + 0.2 * torch.randn(w, device="cuda", generator=g)).half()
        s["residual"] = torch.randn(t, h, w, device="cuda", generator=g).half() * 2 if case["residual"] else None
        if own:
            s["norm"] = q2.RmsNorm(s["weight"], EPS)
            s["sum"] = torch.empty_like(s["residual"]) if case["residual"] else None
            s["y"] = torch.empty(t, h, w, dtype=torch.float16, device="cuda") if case["out"] != "int8" else None
            s["y8"] = torch.empty(t, h, w, dtype=torch.int8, device="cuda") if case["out"] != "fp16" else None
            s["s8"] = torch.empty(t, h, dtype=torch.float32, device="cuda") if case["out"] != "fp16" else None
            s["v8"] = torch.empty(t, h, w, dtype=torch.float16, device="cuda") if case["out"] != "fp16" else None
    elif case["op"] == "int4":
        r, c, n, k = case["rows"], case["cols"], case["tokens"], case["group"]
        s["code"] = torch.randint(0, 256, (r, c // 2), dtype=torch.uint8, device="cuda", generator=g)
        s["scale"] = (0.002 + 0.008 * torch.rand(r, c // k, device="cuda", generator=g)).half()
        s["zero"] = torch.randint(4, 12, (r, c // k), dtype=torch.uint8, device="cuda", generator=g) if case["zeros"] else None
        x = torch.randn(n, c, device="cuda", generator=g)
        if case["x"] == "int8":
            s["xs"] = x.abs().amax(1) / 127
            s["x"] = torch.round(x / s["xs"][:, None]).to(torch.int8)
        else:
            s["x"] = x.half()
        if own:
            zero = None if s["zero"] is None else s["zero"].cpu().numpy()
            s["w"] = q2.Packed(q2.q2_pack_int4(s["code"].cpu().numpy(), s["scale"].cpu().numpy(), zero, k), ntok_max=n)
            s["y"] = torch.empty(n, r, dtype=torch.float16, device="cuda")
    else:
        b, h, d, p = case["batch"], case["kv_heads"], case["dim"], case["page"]
        lens = _lens(case)
        need = [-(-n // p) for n in lens]
        pages = sum(need) + 3
        shape = (pages, p, h, d) if case["order"] == "token" else (pages, h, p, d)
        s["k"], s["v"] = (torch.randn(shape, dtype=torch.float16, device="cuda", generator=g) for _ in range(2))
        if case["order"] == "head":  # stored head by head, seen as [pages][page][heads][dim]
            s["k"], s["v"] = s["k"].transpose(1, 2), s["v"].transpose(1, 2)
        ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        table, at = torch.zeros(b, max(need), dtype=torch.int32, device="cuda"), 0
        for i, m in enumerate(need):
            table[i, :m] = ids[at:at + m]
            at += m
        s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device="cuda")
        # what the qkv projection gives for the new token of each sequence
        hq = h * case["group"]
        s["qkv"] = torch.randn(b, (hq + 2 * h) * d, device="cuda", generator=g).half()
        s["q"] = s["qkv"][:, : hq * d].unflatten(1, (hq, d))
        s["new_k"], s["new_v"] = (s["qkv"][:, a * d: (a + h) * d].unflatten(1, (h, d)) for a in (hq, hq + h))
        if own:
            s["cache"] = q2.PagedKV(s["k"], s["v"], table, q_heads=hq)
            s["o"] = torch.empty(b, hq, d, dtype=torch.float16, device="cuda")
    return s


def run(s):
    case = s["case"]
    if case["op"] == "norm":
        return _norm_own(s) if own else _norm_plain(s)
    if case["op"] == "int4":
        if not own:
            return _int4_plain(s)
        return s["w"].gemv(s["x"], s["y"]) if case["x"] == "fp16" else s["w"].gemv_x8(s["x"], s["xs"], s["y"])
    if not own:
        return _attend_plain(s)
    if not case["append"]:
        return s["cache"].attend(s["q"], s["lens"], out=s["o"])
    return s["cache"].attend(s["q"], s["lens"], new_k=s["new_k"], new_v=s["new_v"], out=s["o"]), s["k"], s["v"]


def _norm_own(s):
    s["norm"].apply(s["x"], residual=s["residual"], residual_out=s["sum"], out=s["y"], out8=s["y8"], scale8=s["s8"])
    res = {"sum": s["sum"], "y": s["y"], "scale": s["s8"]}
    if s["y8"] is not None:
        res["values"] = torch.mul(s["y8"], s["s8"][..., None], out=s["v8"])
    return res


def _norm_plain(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    res = {"sum": h.half() if s["residual"] is not None else None, "y": y.half() if s["case"]["out"] != "int8" else None, "scale": None}
    if s["case"]["out"] != "fp16":
        scale = y.abs().amax(-1, keepdim=True) / 127
        q = torch.round(y / torch.where(scale > 0, scale, torch.ones_like(scale))).clamp(-127, 127)
        res["scale"], res["values"] = scale[..., 0], (q * scale).half()
    return res


def _int4_plain(s):
    code, k = s["code"], s["case"]["group"]
    r, c = code.shape[0], code.shape[1] * 2
    w = torch.stack([code & 15, code >> 4], dim=-1).view(r, c // k, k).float()  # the low four bits are the even column
    w = (w - (8.0 if s["zero"] is None else s["zero"].float()[..., None])) * s["scale"].float()[..., None]
    x = s["x"].float()
    y = x @ w.view(r, c).t()
    return (y if s["case"]["x"] == "fp16" else y * s["xs"][:, None]).half()


def _attend_plain(s):
    case, page = s["case"], s["case"]["page"]
    b, h, g, d = case["batch"], case["kv_heads"], case["group"], case["dim"]
    table, lens = s["table"].long(), s["lens"].long()
    if case["append"]:
        last = lens - 1
        at = table.gather(1, (last // page)[:, None])[:, 0], last % page
        s["k"][at], s["v"][at] = s["new_k"], s["new_v"]
    t = torch.arange(case["length"], device=table.device)
    rows = table[:, t // page], (t % page).expand(b, -1)
    q = s["q"].float().view(b, h, g, d)
    score = torch.einsum("bhgd,blhd->bhgl", q, s["k"][rows].float()) * d ** -0.5
    score = score.masked_fill((t >= lens[:, None])[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    o = torch.einsum("bhgl,blhd->bhgd", p, s["v"][rows].float()) / p.sum(-1, keepdim=True)
    o = o.reshape(b, h * g, d).half()
    return (o, s["k"], s["v"]) if case["append"] else o


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        out = {"sum": None, "y": None, "scale": None}
        hidden = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        y = hidden / (hidden.square().sum(-1, keepdim=True) / case["width"] + EPS).sqrt() * s["weight"].double()
        if s["residual"] is not None:
            out["sum"] = hidden
        if case["out"] != "int8":
            out["y"] = y
        if case["out"] != "fp16":
            top = y.abs().amax(-1)
            out["scale"] = top / 127
            out["values"] = torch.round(y * 127 / top[..., None]) * top[..., None] / 127
        return out
    if case["op"] == "int4":
        x = s["x"].double()
        if case["x"] == "int8":
            x = x * s["xs"].double()[:, None]
        y, k = torch.zeros(case["tokens"], case["rows"], dtype=torch.float64, device="cuda"), case["group"]
        for a in range(case["cols"] // k):  # one group of columns at a time
            part = s["code"][:, a * k // 2: (a + 1) * k // 2].double()
            high = torch.floor(part / 16)
            zero = 8 if s["zero"] is None else s["zero"][:, a: a + 1].double()
            xa = x[:, a * k: (a + 1) * k]
            y += (xa[:, 0::2] @ (part - 16 * high - zero).t() + xa[:, 1::2] @ (high - zero).t()) * s["scale"][:, a].double()
        return y
    d, page, group = case["dim"], case["page"], case["group"]
    out = torch.zeros(case["batch"], case["kv_heads"] * group, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        pages = s["table"][b, : -(-n // page)].long()
        for h in range(case["kv_heads"]):
            k, v = (pool[pages, :, h].reshape(-1, d)[:n].double() for pool in (s["k"], s["v"]))
            if case["append"]:
                k[n - 1], v[n - 1] = s["new_k"][b, h].double(), s["new_v"][b, h].double()
            q = s["q"][b, h * group: (h + 1) * group].double()
            out[b, h * group: (h + 1) * group] = torch.softmax(q @ k.t() / math.sqrt(d), dim=-1) @ v
    return (out, None, None) if case["append"] else out
