"""The key-value cache of a decode step, as cases that can be timed and checked.

``append``   new tokens of every sequence into a paged cache, one each or whole prompts: queries and keys turned by their
             positions' angles on the way, the cache in fp16 or in 4 bits (the rows are then read back as what they stand
             for), and, where asked for, the least and greatest key of every block of 64 tokens kept up.
``attend4``  attention of one new token per sequence over a paged cache held in 4 bits.
``sparse``   attention of one new token per sequence over the blocks of 64 tokens whose bounds promise the most to its
             queries: the selection and the attention over what it selects, from an fp16 or a 4-bit cache.

Four bits: a row's head is cut into groups of 32 or 64 values; a group has an fp16 offset m (its least value) and an fp16
step s (its range / 15), a value is m + s * c with c from 0 to 15, the even column in a byte's low half.

Each has a plain form (elementary operations in 32 bits, in 64 where a value next to a border decides), the library's
form (``own``), and its definition in 64 bits (``exact``).  Heads are those of the Qwen3-8B- and 14B-shaped stacks, and
smaller ones of the tests.
"""
import math

import torch

own = False
BLOCK = 64          # tokens of a block that is selected as one
REACH = 1 << 18     # positions that a table of angles covers at most


def listed():
    return [
        # one sequence early in its answer, 8B heads: latency counts
        {"name": "append 1 token", "op": "append", "batch": 1, "tokens": 1, "past": 776, "bits": 16, "q_group": 4, "kv_heads": 8, "dim": 128, "rot": 128, "style": "half", "group": 64, "page": 16, "order": "token", "bounds": False},
        # 64 sequences decoded together into a 4-bit cache whose blocks are selected from, 14B heads
        {"name": "append 64 tokens 4 bits", "op": "append", "batch": 64, "tokens": 64, "past": 8000, "bits": 4, "q_group": 5, "kv_heads": 8, "dim": 128, "rot": 128, "style": "half", "group": 64, "page": 64, "order": "head", "bounds": True},
        # a few prompts and continued sequences of odd lengths, small heads of which half is turned, pairs side by side
        {"name": "append 5 ragged 3001 4 bits", "op": "append", "batch": 5, "tokens": 3001, "past": 1000, "bits": 4, "q_group": 4, "kv_heads": 2, "dim": 64, "rot": 32, "style": "pairs", "group": 32, "page": 24, "order": "token", "bounds": False},
        # long prompts of four sequences, 8B heads, fp16, bounds kept up
        {"name": "append 4 prompts 16384", "op": "append", "batch": 4, "tokens": 16384, "past": 0, "bits": 16, "q_group": 4, "kv_heads": 8, "dim": 128, "rot": 128, "style": "half", "group": 64, "page": 256, "order": "token", "bounds": True},
        # one sequence early in its answer, 8B heads: latency counts
        {"name": "attend4 1x777", "op": "attend4", "batch": 1, "length": 777, "ragged": False, "kv_heads": 8, "q_group": 4, "dim": 128, "group": 64, "page": 16, "order": "token"},
        # sequences of every length up to 4096 decoded together, 14B heads, small groups
        {"name": "attend4 16 ragged 4096", "op": "attend4", "batch": 16, "length": 4096, "ragged": True, "kv_heads": 8, "q_group": 5, "dim": 128, "group": 32, "page": 16, "order": "head"},
        # a full batch of long sequences, 8B heads, pages stored head by head
        {"name": "attend4 64x8192", "op": "attend4", "batch": 64, "length": 8192, "ragged": False, "kv_heads": 8, "q_group": 4, "dim": 128, "group": 64, "page": 64, "order": "head"},
        # one very long sequence: the work has to be split over its length
        {"name": "attend4 1x131072", "op": "attend4", "batch": 1, "length": 131072, "ragged": False, "kv_heads": 8, "q_group": 4, "dim": 128, "group": 64, "page": 256, "order": "head"},
        # a few sequences that have just outgrown their budget: latency counts
        {"name": "sparse 3x1500 of 8 blocks", "op": "sparse", "batch": 3, "length": 1500, "ragged": True, "bits": 16, "blocks": 8, "first": 1, "kv_heads": 2, "q_group": 4, "dim": 64, "group": 64, "page": 16, "order": "token"},
        # one very long sequence, 8B heads, a thirty-second of it attended
        {"name": "sparse 1x131072 of 64 blocks", "op": "sparse", "batch": 1, "length": 131072, "ragged": False, "bits": 16, "blocks": 64, "first": 1, "kv_heads": 8, "q_group": 4, "dim": 128, "group": 64, "page": 256, "order": "head"},
        # long sequences of every length decoded together from a 4-bit cache, 14B heads
        {"name": "sparse 32 ragged 32768 4 bits", "op": "sparse", "batch": 32, "length": 32768, "ragged": True, "bits": 4, "blocks": 64, "first": 0, "kv_heads": 8, "q_group": 5, "dim": 128, "group": 64, "page": 64, "order": "head"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend4", "sparse"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    heads = {"kv_heads": kv_heads, "q_group": rng.choice([1, 2, 3, 4, 5, 6, 8, 16]), "dim": dim, "group": rng.choice([32, 64]), "order": rng.choice(["token", "head"])}
    if op == "append":
        batch = _log(rng, 1, 256)
        tokens = batch if rng.random() < 0.4 else min(_log(rng, batch, 64 * batch + 1000), 16384 * 6144 // (kv_heads * dim * (heads["q_group"] + 2)), 16384)
        bounds = rng.random() < 0.5
        past = rng.choice([0, _log(rng, 1, min(100000, (1 << 28) // (batch * kv_heads * dim)))])
        return {"op": "append", "batch": min(batch, tokens), "tokens": tokens, "past": past, "bits": rng.choice([16, 4]), **heads,
                "rot": rng.choice([dim, dim // 2, 32]), "style": rng.choice(["half", "pairs"]), "page": rng.choice([16, 32, 64, 256] if bounds else [8, 16, 24, 64, 100, 256]), "bounds": bounds}
    batch = _log(rng, 1, 64)
    length = _log(rng, 1, min(131072, 64 * 8192 * 8 * 128 // (batch * kv_heads * dim)))
    if op == "attend4":
        return {"op": "attend4", "batch": batch, "length": length, "ragged": rng.random() < 0.5, **heads, "page": rng.choice([8, 16, 24, 32, 64, 100, 256])}
    return {"op": "sparse", "batch": batch, "length": length, "ragged": rng.random() < 0.5, "bits": rng.choice([16, 4]), "blocks": _log(rng, 2, 256), "first": rng.choice([0, 1]), **heads,
            "page": rng.choice([16, 32, 64, 128, 256])}


def _spread(n, most, ragged):
    """`n` lengths: all `most`, or spread from 1 to `most`."""
    if not ragged or n == 1:
        return [most] * n
    return [1 + (most - 1) * ((i * 29 + n - 1) % n) // (n - 1) for i in range(n)]


def _counts(case):
    """New tokens of each sequence (one at least): one each, or uneven shares."""
    b, n = case["batch"], case["tokens"]
    weight = [1 + i * 7 % 5 for i in range(b)]
    got = [1 + (n - b) * w // sum(weight) for w in weight]
    got[b // 2] += n - sum(got)
    return got


def _lens(case):
    if case["op"] != "append":
        return _spread(case["batch"], case["length"], case["ragged"])
    past = _spread(case["batch"], case["past"], True) if case["past"] else [0] * case["batch"]
    return [p + n for p, n in zip(past, _counts(case))]


def _row_bytes(case, bits):
    """Bytes of a key's or a value's row, all heads."""
    d = case["kv_heads"] * case["dim"]
    return 2 * d if bits == 16 else d // 2 + 4 * d // case["group"]


def work(case):
    lens, kv, page, b = _lens(case), case["kv_heads"] * case["dim"], case["page"], case["batch"]
    q = kv * case["q_group"]
    if case["op"] == "append":
        n = case["tokens"]
        # queries in and out, keys and values in, the cache's rows out, as numbers too where they are 4 bits; angles, page numbers
        moved = n * (4 * q + 4 * kv + 2 * _row_bytes(case, case["bits"]) + (4 * kv if case["bits"] == 4 else 0) + 4 * case["rot"]) + 4 * sum(-(-m // page) for m in _counts(case))
        touched = sum((m - 1) // BLOCK - (m - c) // BLOCK + 1 for m, c in zip(lens, _counts(case)))
        return {"bytes": moved + (touched * 4 * kv if case["bounds"] else 0), "flops": 3 * n * (q + kv) * case["rot"] // case["dim"]}
    if case["op"] == "attend4":
        tokens = sum(lens)
        return {"bytes": 2 * tokens * _row_bytes(case, 4) + 4 * b * q + 4 * sum(-(-m // page) for m in lens), "flops": 4 * tokens * q}
    blocks = [-(-m // BLOCK) for m in lens]
    read = sum(min(m, case["blocks"] * BLOCK) for m in lens)
    return {"bytes": sum(blocks) * 4 * kv + 2 * read * _row_bytes(case, case["bits"]) + 4 * b * q + 4 * b * case["kv_heads"] * case["blocks"] + 4 * sum(-(-m // page) for m in lens),
            "flops": 2 * sum(blocks) * q + 4 * read * q}


# ---------------------------------------------------------------- inputs


def _angles(case, device="cuda"):
    """cos and sin of every position's angles, [positions][rot / 2][2] in fp32, made in 64 bits."""
    turn = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=device) / case["rot"])
    at = torch.arange(min(REACH, max(_lens(case))), dtype=torch.float64, device=device)[:, None] * turn
    return torch.stack([at.cos(), at.sin()], dim=-1).float()


def _quantise(x, group):
    """Groups of `group` values along the last axis in 4 bits: codes as numbers [..][groups][group], (step, offset) fp16 [..][groups][2]."""
    x = x.unflatten(-1, (-1, group))
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    m, s = low.half(), ((high - low) / 15).half()
    c = torch.round((x - m.float()) / torch.where(s > 0, s, torch.ones_like(s)).float()).clamp(0, 15)
    return torch.where(s > 0, c, torch.zeros_like(c)), torch.cat([s, m], dim=-1)


def _pack(codes):
    """Codes [..][groups][group] as bytes [..][groups * group / 2], the even column in the low half."""
    c = codes.flatten(-2).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _values(packed, steps):
    """What bytes [..][dim / 2] with (step, offset) [..][groups][2] stand for, in fp32."""
    c = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2).unflatten(-1, (steps.shape[-2], -1)).float()
    return (c * steps[..., :1].float() + steps[..., 1:].float()).flatten(-2)


def _ordered(t, order):
    """The tensor [pages][page][heads][..] stored head by head, or as it is."""
    return t.transpose(1, 2).contiguous().transpose(1, 2) if order == "head" else t


def _bounds_shape(case, pages):
    return (pages, -(-case["page"] // BLOCK), case["kv_heads"], 2, case["dim"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    b, h, d, p = case["batch"], case["kv_heads"], case["dim"], case["page"]
    hq, lens = h * case["q_group"], _lens(case)
    need = [-(-n // p) for n in lens]
    pages = sum(need) + 3
    ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    column = torch.arange(max(need), device="cuda")[None, :]
    many = torch.tensor(need, device="cuda")[:, None]
    table = ids[((many.cumsum(0) - many) + torch.minimum(column, many - 1))].contiguous()
    s = {"case": case, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    if case["op"] == "append":
        n = case["tokens"]
        # what the qkv projection gives for the new tokens; a few columns of the keys far larger than the rest, as keys have
        s["qkv"] = torch.randn(n, (hq + 2 * h) * d, device="cuda", generator=g).half()
        big = torch.rand(h * d, device="cuda", generator=g) < 0.02
        s["qkv"][:, hq * d: (hq + h) * d] *= torch.where(big, 6.0, 1.0).half()
        s["q"], s["new_k"], s["new_v"] = (s["qkv"][:, a * d: (a + m) * d].unflatten(1, (m, d)) for a, m in ((0, hq), (hq, h), (hq + h, h)))
        s["starts"] = None if n == b else torch.tensor([0] + _counts(case), device="cuda").cumsum(0).to(torch.int32)
        s["angles"] = _angles(case)
        shape = (pages, p, h, d)
        if case["bits"] == 16:
            s["k"], s["v"] = (_ordered(torch.zeros(shape, dtype=torch.float16, device="cuda"), case["order"]) for _ in range(2))
        else:
            for name in ("k", "v"):
                s[name] = _ordered(torch.zeros(shape[:3] + (d // 2,), dtype=torch.uint8, device="cuda"), case["order"])
                s[name + "s"] = _ordered(torch.zeros(shape[:3] + (d // case["group"], 2), dtype=torch.float16, device="cuda"), case["order"])
        # blocks that hold tokens already have bounds
        s["bounds"] = torch.randn(_bounds_shape(case, pages), device="cuda", generator=g).half().sort(dim=3).values if case["bounds"] else None
        s["turned"] = torch.empty(n, hq, d, dtype=torch.float16, device="cuda")
        s["out_k"], s["out_v"] = (torch.empty(n, h, d, dtype=torch.float16, device="cuda") for _ in range(2))
    else:
        s["q"] = torch.randn(b, (hq + 2 * h) * d, device="cuda", generator=g).half()[:, : hq * d].unflatten(1, (hq, d))
        sparse = case["op"] == "sparse"
        bits = case.get("bits", 4)
        dt = torch.float16
        s["k"], s["v"] = (_ordered(torch.empty((pages, p, h, d if bits == 16 else d // 2), dtype=dt if bits == 16 else torch.uint8, device="cuda"), case["order"]) for _ in range(2))
        if bits == 4:
            s["ks"], s["vs"] = (_ordered(torch.empty((pages, p, h, d // case["group"], 2), dtype=dt, device="cuda"), case["order"]) for _ in range(2))
        keys = torch.empty((pages, p, h, d), dtype=dt, device="cuda") if sparse else None
        step = max(1, (1 << 26) // (p * h * d))  # pages at a time
        # keys drift along the cache, so that blocks differ; a few columns far larger than the rest
        big = torch.where(torch.rand(h, d, device="cuda", generator=g) < 0.02, 4.0, 1.0)
        for name in ("k", "v"):
            for a in range(0, pages, step):
                m = min(step, pages - a)
                x = torch.randn(m, p, h, d, device="cuda", generator=g)
                if name == "k":
                    x = (x * 0.7 + torch.randn(m, 1, h, d, device="cuda", generator=g) * 0.7) * big
                x = x.half()
                if name == "k" and sparse:
                    keys[a: a + m] = x
                if bits == 16:
                    s[name][a: a + m] = x
                else:
                    codes, steps = _quantise(x.float(), case["group"])
                    s[name][a: a + m], s[name + "s"][a: a + m] = _pack(codes), steps
        if sparse:
            s["bounds"] = torch.zeros(_bounds_shape(case, pages), dtype=dt, device="cuda")
            if p >= BLOCK:
                rows = keys.unflatten(1, (-1, BLOCK))
                s["bounds"].copy_(torch.stack([rows.amin(2), rows.amax(2)], dim=3))
            else:  # a block lies in several pages, its bounds at the first; pages that do not exist repeat the last
                per = BLOCK // p
                wide = table.long()[:, torch.arange(-(-max(need) // per) * per, device="cuda").clamp(max=max(need) - 1)].unflatten(1, (-1, per))
                for i in range(b):
                    rows = keys[wide[i]].flatten(1, 2)
                    s["bounds"][wide[i, :, 0], 0] = torch.stack([rows.amin(1), rows.amax(1)], dim=2)
        del keys
        s["o"] = torch.empty(b, hq, d, dtype=dt, device="cuda")
        s["sel"] = torch.empty(b, h, case["blocks"], dtype=torch.int32, device="cuda") if sparse else None
    if own:
        import dequant_gemv_q2_gb300 as q2
        q2.load()
        if "ks" in s:
            s["cache"] = q2.PagedKV4(s["k"], s["ks"], s["v"], s["vs"], table, q_heads=hq, bounds=s.get("bounds"))
        else:
            s["cache"] = q2.PagedKV(s["k"], s["v"], table, q_heads=hq, bounds=s.get("bounds"))
        if case["op"] == "append":
            s["rope"] = q2.Rope(s["angles"], interleaved=case["style"] == "pairs")
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    op = s["case"]["op"]
    if op == "append":
        return _append_own(s) if own else _append_plain(s)
    if op == "attend4":
        return s["cache"].attend(s["q"], s["lens"], out=s["o"]) if own else _attend4_plain(s)
    return _sparse_own(s) if own else _sparse_plain(s)


def _append_own(s):
    s["cache"].append(s["new_k"], s["new_v"], s["lens"], starts=s["starts"], q=s["q"], q_out=s["turned"], rope=s["rope"])
    if s["case"]["bits"] == 16:
        return {"q": s["turned"], "k": s["k"], "v": s["v"], "bounds": s["bounds"]}
    s["cache"].read(s["lens"], starts=s["starts"], k_out=s["out_k"], v_out=s["out_v"])
    return {"q": s["turned"], "k": s["out_k"], "v": s["out_v"], "bounds": s["bounds"]}


def _sparse_own(s):
    case = s["case"]
    sel = s["cache"].select(s["q"], s["lens"], case["blocks"], first=case["first"], out=s["sel"])
    return {"sel": sel, "o": s["cache"].attend(s["q"], s["lens"], blocks=sel, out=s["o"])}


def _turn(x, angles, style):
    """The first columns of every head turned, in 64 bits, rounded to 32."""
    rot = angles.shape[1] * 2
    cos, sin = angles.double().unsqueeze(1).unbind(-1)
    y, rest = x[..., :rot].double(), x[..., rot:].float()
    if style == "half":
        a, c = y.chunk(2, dim=-1)
        y = torch.cat([a * cos - c * sin, c * cos + a * sin], dim=-1)
    else:
        a, c = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - c * sin, c * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([y.float(), rest], dim=-1)


def _append_plain(s):
    case, page, table, lens = s["case"], s["case"]["page"], s["table"].long(), s["lens"].long()
    n = case["tokens"]
    row = torch.arange(n, device=table.device)
    starts = s["starts"].long() if s["starts"] is not None else torch.arange(n + 1, device=table.device)
    b = torch.searchsorted(starts, row, right=True) - 1
    pos = lens[b] - (starts[b + 1] - row)
    at = table[b, pos // page], pos % page
    angles = s["angles"][pos]
    turned = _turn(s["q"], angles, case["style"]).half()
    k, v = _turn(s["new_k"], angles, case["style"]), s["new_v"].float()
    out = {"q": turned, "bounds": s["bounds"]}
    if case["bits"] == 16:
        s["k"][at], s["v"][at] = k.half(), v.half()
        out["k"], out["v"] = s["k"], s["v"]
    else:
        for name, x in (("k", k), ("v", v)):
            codes, steps = _quantise(x, case["group"])
            s[name][at], s[name + "s"][at] = _pack(codes), steps
            out[name] = _values(s[name][at], s[name + "s"][at]).half()
    if case["bounds"]:
        begin = pos // BLOCK * BLOCK
        block = table[b, begin // page] * s["bounds"].shape[1] + begin % page // BLOCK
        flat = s["bounds"].flatten(0, 1).float()
        new = torch.zeros(flat.shape[0], device=table.device).index_add_(0, block, (pos == begin).float())[:, None, None] > 0  # blocks that begin here
        low, high = flat.unbind(2)
        low, high = low.masked_fill(new, math.inf), high.masked_fill(new, -math.inf)
        key = k.half().float()
        s["bounds"].copy_(torch.stack([low.index_reduce_(0, block, key, "amin"), high.index_reduce_(0, block, key, "amax")], dim=2).view_as(s["bounds"]))
    return out


def _attend(q, k, v, live):
    """Attention of q [b][h][g][d] over k, v [b][h][l][d] where `live` [b][h][l], in fp32; zeros where nothing is."""
    score = torch.einsum("bhgd,bhld->bhgl", q, k) * q.shape[-1] ** -0.5
    score = score.masked_fill(~live[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgl,bhld->bhgd", p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.flatten(1, 2).half()


def _attend4_plain(s):
    case, page = s["case"], s["case"]["page"]
    table, lens = s["table"].long(), s["lens"].long()
    t = torch.arange(case["length"], device=table.device)
    rows = table[:, t // page], (t % page).expand(case["batch"], -1)
    k, v = (_values(s[n][rows], s[n + "s"][rows]).transpose(1, 2) for n in ("k", "v"))
    live = (t < lens[:, None])[:, None].expand(-1, case["kv_heads"], -1)
    return _attend(s["q"].float().unflatten(1, (case["kv_heads"], -1)), k, v, live)


def _sparse_plain(s):
    case, page, most = s["case"], s["case"]["page"], s["case"]["blocks"]
    table, lens = s["table"].long(), s["lens"].long()
    q = s["q"].unflatten(1, (case["kv_heads"], -1))
    blocks = -(-lens // BLOCK)
    i = torch.arange(-(-case["length"] // BLOCK), device=table.device)
    begin = i * BLOCK
    low, high = s["bounds"][table[:, begin // page], (begin % page // BLOCK).expand(case["batch"], -1)].double().unbind(3)  # [b][blocks][h][d]
    # the most that any key within the bounds could give, the largest over the head's queries, in 64 bits and rounded to 32
    score = torch.einsum("bhgd,bnhd->bhgn", q.double().clamp(min=0), high) + torch.einsum("bhgd,bnhd->bhgn", q.double().clamp(max=0), low)
    score = score.float().amax(2)
    last = blocks[:, None, None]
    kept = (i < case["first"]) | (i == last - 1)
    score = score.masked_fill(kept, math.inf).masked_fill(i >= last, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :most]
    best = torch.where(best < last, best, torch.full_like(best, 1 << 30)).sort(dim=-1).values
    best = torch.nn.functional.pad(best, (0, most - best.shape[-1]), value=1 << 30)
    there = best < (1 << 30)
    # the selected tokens
    t = (best[..., None] * BLOCK + torch.arange(BLOCK, device=table.device)).flatten(2)
    live = (t < lens[:, None, None]) & there.repeat_interleave(BLOCK, dim=-1)
    t = torch.where(live, t, torch.zeros_like(t))
    rows = table[torch.arange(case["batch"], device=table.device)[:, None, None], t // page], t % page, torch.arange(case["kv_heads"], device=table.device)[:, None]
    k, v = (s[n][rows].float() if case["bits"] == 16 else _values(s[n][rows], s[n + "s"][rows]) for n in ("k", "v"))
    return {"sel": torch.where(there, best, torch.full_like(best, -1)).to(torch.int32), "o": _attend(q.float(), k, v, live)}


# ---------------------------------------------------------------- the definitions in 64 bits


def _rows64(s, name, pages, slots, head):
    """Rows of one head as they stand in the cache, in 64 bits."""
    rows = s[name][pages, slots, head]
    if name + "s" not in s:
        return rows.double()
    steps, byte = s[name + "s"][pages, slots, head].double().repeat_interleave(s["case"]["group"], dim=-2), rows.double()
    code = torch.empty_like(steps[..., 0])
    code[..., 1::2] = torch.floor(byte / 16)
    code[..., 0::2] = byte - 16 * code[..., 1::2]
    return steps[..., 1] + steps[..., 0] * code


def exact(case, seed):
    s = prepare(case, seed)
    page, d, heads, group = case["page"], case["dim"], case["kv_heads"], case["q_group"]
    lens = _lens(case)
    if case["op"] == "append":
        return _append_exact(s)
    out = torch.zeros(case["batch"], heads * group, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        for h in range(heads):
            q = s["q"][b, h * group: (h + 1) * group].double()
            at = torch.arange(n, device="cuda")
            if case["op"] == "sparse":
                count = (n + BLOCK - 1) // BLOCK
                first = torch.arange(count, device="cuda") * BLOCK
                bound = s["bounds"][s["table"][b].long()[first // page], first % page // BLOCK, h].double()
                best = torch.maximum(q[:, None] * bound[None, :, 0], q[:, None] * bound[None, :, 1]).sum(-1).float().amax(0)
                best[: case["first"]] = math.inf
                best[count - 1] = math.inf
                taken = torch.sort(best, descending=True, stable=True).indices[: case["blocks"]]
                at = at[torch.isin(at // BLOCK, taken)]
            pages = s["table"][b].long()[at // page]
            k, v = (_rows64(s, name, pages, at % page, h) for name in ("k", "v"))
            out[b, h * group: (h + 1) * group] = torch.softmax(q @ k.t() / math.sqrt(d), dim=-1) @ v
    return {"sel": None, "o": out} if case["op"] == "sparse" else out


def _append_exact(s):
    case, d, rot = s["case"], s["case"]["dim"], s["case"]["rot"]
    counts = _counts(case)
    pos = torch.cat([torch.arange(n - c, n, device="cuda") for n, c in zip(_lens(case), counts)])
    owner = torch.cat([torch.full((c,), i, device="cuda") for i, c in enumerate(counts)])

    def turned(x):
        y = x.double().clone()
        for i in range(rot // 2):
            a, b = (i, i + rot // 2) if case["style"] == "half" else (2 * i, 2 * i + 1)
            cos, sin = (s["angles"][pos, i, j].double()[:, None] for j in (0, 1))
            y[..., a] = x[..., a].double() * cos - x[..., b].double() * sin
            y[..., b] = x[..., b].double() * cos + x[..., a].double() * sin
        return y

    k = turned(s["new_k"])
    out = {"q": turned(s["q"]), "k": None, "v": None, "bounds": None}
    page = s["table"].long()[owner, pos // case["page"]]
    for name, x in (("k", k), ("v", s["new_v"].double())):
        if case["bits"] == 16:
            pool = s[name].double()
            pool[page, pos % case["page"]] = x
            out[name] = pool
        else:
            y = x.float().double().unflatten(-1, (d // case["group"], case["group"]))
            low = y.min(dim=-1, keepdim=True).values
            step = ((y.max(dim=-1, keepdim=True).values - low) / 15).half().double()
            low = low.half().double()
            code = torch.where(step > 0, torch.round((y - low) / step.clamp(min=1e-30)), 0.0).clamp(0, 15)
            out[name] = (low + step * code).flatten(-2)
    if case["bounds"]:
        kept = s["bounds"].double()
        block = pos // BLOCK
        place = s["table"].long()[owner, block * BLOCK // case["page"]] * kept.shape[1] + block * BLOCK % case["page"] // BLOCK
        flat, key = kept.flatten(0, 1), k.half().double()
        for i in torch.unique(place).tolist() if case["tokens"] <= 20000 else []:
            rows = key[place == i]
            low, high = rows.min(0).values, rows.max(0).values
            if not (pos[place == i] % BLOCK == 0).any():
                low, high = torch.minimum(low, flat[i, :, 0]), torch.maximum(high, flat[i, :, 1])
            flat[i] = torch.stack([low, high], dim=1)
        out["bounds"] = flat.view(kept.shape)
    return out
