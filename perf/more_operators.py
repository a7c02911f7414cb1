"""Measured cases of rotary positions with several axes, attention over a shared prefix, and attention over selected
blocks of a paged cache.

``run`` computes one pass of an operator: with ``own`` false in elementary torch operations, with ``own`` true through
the package's entry points.  ``exact`` gives the same outputs in 64 bits.
"""

import math

import torch

own = False

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16,
         "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2, "e4m3": 1, "int8": 1}
TOP = {"e4m3": 448.0, "int8": 127.0}
BASE = 500000.0


# ---------------------------------------------------------------------------------- cases
def listed():
    return [
        # the gradient of an image encoder's queries: rows and columns of odd-sized pictures, each with its own frequencies
        {"name": "axes gradient", "op": "axes", "type": "fp32", "batch": 3, "seq": 1023, "heads": 16, "dim": 80, "rot": 80,
         "axes": 2, "order": "blocks", "own": True, "pairs": "interleaved", "split": False, "backward": True},
        # the queries of a batch of videos: time, height and width share the frequencies in turn; heads split on the way
        {"name": "axes prompt", "op": "axes", "type": "bf16", "batch": 8, "seq": 8192, "heads": 32, "dim": 128, "rot": 128,
         "axes": 3, "order": "cyclic", "own": False, "pairs": "half", "split": True, "backward": False},
        # the new tokens of 64 conversations, keys turned as they are stored, some rows padding
        {"name": "axes write step", "op": "write", "type": "bf16", "kind": "bf16", "tokens": 64, "heads": 8, "dim": 128,
         "rot": 128, "axes": 3, "order": "blocks", "own": False, "pairs": "half", "page": 16, "layout": "tokens", "pad": 5},
        # a video's prompt of odd length into an 8-bit cache
        {"name": "axes write prompt", "op": "write", "type": "bf16", "kind": "e4m3", "tokens": 16389, "heads": 8, "dim": 128,
         "rot": 128, "axes": 3, "order": "cyclic", "own": False, "pairs": "half", "page": 64, "layout": "heads", "pad": 0},
        # four answers to one short prompt: latency
        {"name": "prefix few", "op": "prefix", "type": "bf16", "kind": "bf16", "batch": 4, "prefix": 1000, "length": 60,
         "heads": 32, "kv": 8, "dim": 128, "page": 16, "layout": "tokens", "empty": False},
        # an ordinary serving batch behind a long instruction, one slot without tokens of its own
        {"name": "prefix batch", "op": "prefix", "type": "bf16", "kind": "bf16", "batch": 32, "prefix": 8191, "length": 1024,
         "heads": 32, "kv": 8, "dim": 128, "page": 16, "layout": "tokens", "empty": True},
        # questions about one long document held in 8 bits
        {"name": "prefix codes", "op": "prefix", "type": "fp16", "kind": "e4m3", "batch": 24, "prefix": 65536, "length": 300,
         "heads": 32, "kv": 4, "dim": 96, "page": 32, "layout": "heads", "empty": False},
        # many samples of one long prompt: the scores are a large matrix product
        {"name": "prefix large", "op": "prefix", "type": "bf16", "kind": "bf16", "batch": 128, "prefix": 32768, "length": 2048,
         "heads": 64, "kv": 8, "dim": 128, "page": 16, "layout": "heads", "empty": False},
        # one step of a serving batch: the newest token's block gets its key, then each cache head's blocks are chosen
        {"name": "choose step", "op": "choose", "type": "bf16", "kind": "bf16", "batch": 16, "length": 32768, "spread": True,
         "new": False, "heads": 32, "kv": 8, "dim": 128, "page": 64, "layout": "heads", "count": 64, "first": 1, "last": 2},
        # the first step behind two long prompts: the keys of all their blocks, small ones
        {"name": "choose prompt", "op": "choose", "type": "bf16", "kind": "e4m3", "batch": 2, "length": 131071, "spread": False,
         "new": True, "heads": 64, "kv": 8, "dim": 128, "page": 16, "layout": "tokens", "count": 256, "first": 4, "last": 16},
        # one user, 4096 tokens chosen out of a long context: latency
        {"name": "attend chosen", "op": "attend", "type": "bf16", "kind": "bf16", "batch": 1, "length": 131072, "spread": False,
         "heads": 32, "kv": 8, "dim": 128, "page": 64, "layout": "heads", "count": 64},
        # a serving batch, 4096 tokens of each sequence in small blocks
        {"name": "attend chosen batch", "op": "attend", "type": "bf16", "kind": "bf16", "batch": 64, "length": 16384,
         "spread": True, "heads": 64, "kv": 8, "dim": 128, "page": 16, "layout": "tokens", "count": 256},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["axes", "write", "prefix", "prefix", "choose", "attend"])
    dim = rng.choice([32, 64, 72, 80, 96, 112, 128, 128, 160, 192, 256])
    if op in ("axes", "write"):
        order = rng.choice(["blocks", "cyclic"])
        rot = dim if order == "cyclic" else rng.choice([dim, dim, dim // 2 // 4 * 4])
        c = {"op": op, "type": rng.choice(["bf16", "fp16", "fp32"]), "heads": rng.choice([1, 4, 8, 20, 32]), "dim": dim, "rot": rot,
             "axes": rng.choice([2, 3, 3, 4]), "order": order, "own": rng.random() < 0.4, "pairs": rng.choice(["half", "interleaved"])}
        if op == "axes":
            c.update(batch=rng.randint(1, 16), seq=_log(rng, 1, 8192), split=rng.random() < 0.5, backward=rng.random() < 0.5)
            while c["batch"] * c["seq"] * c["heads"] * dim * BYTES[c["type"]] > 1 << 29:
                c["seq"] = c["seq"] // 2
            return c
        c.update(kind=rng.choice([c["type"], "e4m3"]), tokens=_log(rng, 1, 60000), page=rng.choice([8, 16, 16, 32, 64, 128]),
                 layout=rng.choice(["tokens", "heads"]), pad=rng.choice([0, 0, 3]))
        while c["tokens"] * c["heads"] * dim > 1 << 26:
            c["tokens"] = c["tokens"] // 2
        c["pad"] = c["pad"] if c["tokens"] > 8 else 0
        return c
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32", "e4m3", "int8"])
    c = {"op": op, "type": kind if kind in ("bf16", "fp16", "fp32") else rng.choice(["bf16", "fp16"]), "kind": kind,
         "kv": rng.choice([1, 2, 4, 8, 8]), "dim": dim, "page": rng.choice([8, 16, 16, 32, 64, 128]),
         "layout": rng.choice(["tokens", "heads"])}
    c["heads"] = c["kv"] * rng.choice([1, 2, 4, 5, 7, 8])
    if op == "prefix":
        c.update(batch=_log(rng, 1, 128), prefix=_log(rng, 1, 60000), length=_log(rng, 1, 2048), empty=rng.random() < 0.3)
        while c["batch"] * c["heads"] * c["prefix"] * dim > 1 << 35 or c["prefix"] * c["kv"] * dim > 1 << 28:
            c["prefix"] = c["prefix"] // 2
        while c["batch"] * c["length"] * c["kv"] * dim * BYTES[kind] > 1 << 28:
            c["length"] = c["length"] // 2
        return c
    c.update(batch=_log(rng, 1, 64), length=_log(rng, 1, 131072), spread=rng.random() < 0.7)
    while c["batch"] * c["length"] * c["kv"] * dim * BYTES[kind] > 1 << 29:
        c["length"] = c["length"] // 2
    c["count"] = _log(rng, 8, 4096 // c["page"] if c["page"] < 128 else 32)
    if op == "choose":
        c.update(first=rng.choice([0, 1, 4]), last=rng.choice([1, 2, 4]), new=rng.random() < 0.4)
    return c


# ---------------------------------------------------------------------------------- shapes
def _lens(c):
    """Lengths of a batch: all the same, or spread evenly below the longest (the golden ratio's multiples)."""
    n = [c["length"]] * c["batch"]
    if c.get("spread", True):
        n = [max(1, round(c["length"] * (1 - (i * 0.6180339887498949) % 1))) for i in range(c["batch"])]
    if c.get("empty") and c["batch"] > 1:
        n[-1] = 0
    return n


def _sections(c):
    """Pairs of each axis: the first has what the others leave."""
    pairs, axes = c["rot"] // 2, c["axes"]
    each = pairs // axes
    return [pairs - (axes - 1) * each] + [each] * (axes - 1)


def _frequencies(c, device):
    """(axis of each pair, its angle per position in 64 bits)."""
    pairs, axes, sections = c["rot"] // 2, c["axes"], _sections(c)
    i = torch.arange(pairs, device=device)
    if c["order"] == "blocks":
        ends = torch.tensor(sections, device=device).cumsum(0)
        axis = (i[:, None] >= ends).sum(1)
    else:  # pair i is axis i mod axes as long as that one has pairs left, else the first
        axis = i % axes
        axis = torch.where(i < axes * torch.tensor(sections, device=device)[axis], axis, torch.zeros_like(axis))
    if not c["own"]:
        return axis, BASE ** (-2 * i.double() / c["rot"])
    within = torch.nn.functional.one_hot(axis, axes).cumsum(0).gather(1, axis[:, None])[:, 0] - 1
    return axis, BASE ** (-within.double() / torch.tensor(sections, device=device)[axis])


# ---------------------------------------------------------------------------------- inputs
def _randn(gen, shape, dtype, device):
    return torch.randn(shape, generator=gen, device=device, dtype=torch.float32).to(dtype)


def _pool(c, pages):
    """The shape (pages, ...) of a cache tensor and of its scales, and the layout text of each."""
    h, p, d = c.get("kv", c["heads"]), c["page"], c["dim"]
    if c["layout"] == "tokens":
        return ((pages, p, h, d), (pages, p, h), f"({d},{h},{p},{pages}):(1,{d},{h * d},{p * h * d})",
                f"({h},{p},{pages}):(1,{h},{p * h})")
    return ((pages, h, p, d), (pages, h, p), f"({d},{h},{p},{pages}):(1,{p * d},{d},{h * p * d})",
            f"({h},{p},{pages}):({p},1,{h * p})")


def _filled(gen, c, shape, device):
    """A cache tensor that holds values, and its scales."""
    if c["kind"] not in TOP:
        return _randn(gen, shape, TYPES[c["kind"]], device), None
    x = torch.randn(shape, generator=gen, device=device, dtype=torch.float32)
    scale = x.abs().amax(-1) / TOP[c["kind"]]
    x = x / scale.unsqueeze(-1)
    return (x.to(torch.float8_e4m3fn) if c["kind"] == "e4m3" else x.round().to(torch.int8)), scale


def _positions(gen, c, tokens, device):
    """(axes, tokens): a frame's number, and rows and columns inside it; the first picture starts anywhere."""
    first = torch.randint(0, 4096, (c["axes"], 1), generator=gen, device=device)
    t = torch.arange(tokens, device=device)
    side = 24
    grid = torch.stack([t // (side * side), t // side % side, t % side, t // 7])[:c["axes"]]
    return (first + grid).contiguous()


def prepare(case, seed):
    c = case
    device = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    s = {"case": c, "device": device}
    t = TYPES[c["type"]]
    h, d = c["heads"], c["dim"]
    if c["op"] == "axes":
        b, n = c["batch"], c["seq"]
        s["x"] = _randn(gen, (b, n, h, d), t, device)
        s["positions"] = _positions(gen, c, b * n, device)
        s["y"] = torch.empty((b, h, n, d) if c["split"] else (b, n, h, d), dtype=t, device=device)
    elif c["op"] == "write":
        n = c["tokens"]
        pages = -(-n // c["page"]) + 3
        shape, scales, _, _ = _pool(c, pages)
        # pages come from a free list in no order, the tokens of a page follow each other
        free = torch.randperm(pages, generator=gen, device=device)
        at = torch.arange(n, device=device)
        s["slots"] = free[at // c["page"]] * c["page"] + at % c["page"]
        if c["pad"]:
            s["slots"][torch.randperm(n, generator=gen, device=device)[:c["pad"]]] = -1
        s["k"], s["v"] = _randn(gen, (n, h, d), t, device), _randn(gen, (n, h, d), t, device)
        s["ck"], s["cv"] = (torch.zeros(shape, dtype=torch.uint8, device=device).view(TYPES["e4m3"]) if c["kind"] == "e4m3"
                            else torch.zeros(shape, dtype=TYPES[c["kind"]], device=device) for _ in range(2))
        s["ks"], s["vs"] = (torch.zeros(scales, device=device) if c["kind"] in TOP else None for _ in range(2))
        s["positions"] = _positions(gen, c, n, device)
    else:
        b, p = c["batch"], c["page"]
        lens = _lens(c)
        need = [-(-n // p) for n in lens]
        shared = -(-c["prefix"] // p) if c["op"] == "prefix" else 0
        pages, width = sum(need) + shared + 3, max(max(need), 1)
        shape, _, _, _ = _pool(c, pages)
        (s["ck"], s["ks"]), (s["cv"], s["vs"]) = _filled(gen, c, shape, device), _filled(gen, c, shape, device)
        free = torch.randperm(pages, generator=gen, device=device, dtype=torch.int32)
        table = torch.zeros((b, width), dtype=torch.int32, device=device)
        at = shared
        for i, n in enumerate(need):
            table[i, :n] = free[at:at + n]
            at += n
        s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=device)
        s["q"] = _randn(gen, (b, h, d), t, device)
        if c["op"] == "prefix":
            s["prefix"] = free[:shared].clone()
            s["prefix_len"] = torch.tensor([c["prefix"]], dtype=torch.int32, device=device)
        if c["op"] == "choose":
            s["keys"] = torch.zeros((pages, c["kv"], d), dtype=t, device=device)
            s["spare"] = int(free[-1])  # a page that no sequence has
            if not c["new"]:  # the keys of all earlier blocks
                page = torch.arange(pages, device=device)
                s["keys"][page] = _mean(c, s, page, torch.full_like(page, p)).to(t)
            seq = torch.repeat_interleave(torch.arange(b, device=device), torch.tensor(lens, device=device))
            pos = torch.cat([torch.arange(n, device=device) for n in lens])
            if not c["new"]:  # the newest token of each sequence
                seq, pos = torch.arange(b, device=device), s["lens"].long() - 1
            s["slots"] = table.long()[seq, pos // p] * p + pos % p
            s["blocks"] = torch.empty((b, c["kv"], c["count"]), dtype=torch.int32, device=device)
        else:
            s["out"] = torch.empty((b, h, d), dtype=t, device=device)
            s["lse"] = torch.empty((b, h), dtype=torch.float32, device=device)
        if c["op"] == "attend":  # blocks that a score chose: any, the last among them, in their order
            count = torch.tensor(need, device=device)[:, None, None]
            score = torch.rand((b, c["kv"], width), generator=gen, device=device)
            j = torch.arange(width, device=device)
            score = torch.where(j == count - 1, 2.0, score).masked_fill(j >= count, -1.0)
            top = torch.sort(score, dim=-1, descending=True).indices[..., :c["count"]]
            top = torch.where(score.gather(-1, top) < 0, width, top).sort(-1).values
            s["blocks"] = torch.full((b, c["kv"], c["count"]), -1, dtype=torch.int32, device=device)
            s["blocks"][..., :top.shape[-1]] = torch.where(top == width, -1, top).int()
    if own:
        _handles(c, s)
    return s


def _handles(c, s):
    """What a user of the package keeps: parsed layouts, the table of frequencies, the cache's description, a workspace."""
    import layout_remapping_copy_amd as lr

    s["lr"] = lr
    d, h = c["dim"], c["heads"]
    if c["op"] in ("axes", "write"):
        s["rope"] = lr.rope_axes_table(c["rot"], _sections(c), order=c["order"], own=c["own"], base=BASE, device=s["device"])
    if c["op"] == "axes":
        b, n = c["batch"], c["seq"]
        s["Lx"] = lr.Layout(f"({d},{h},({n},{b})):(1,{d},({h * d},{n * h * d}))")
        s["Ly"] = lr.Layout(f"({d},{h},({n},{b})):(1,{n * d},({d},{n * h * d}))") if c["split"] else s["Lx"]
        return
    pages = s["ck"].shape[0]
    _, _, layout, scales = _pool(c, pages)
    s["cache"] = lr.PagedCache(s["ck"], layout, s["cv"], layout, s["ks"], s["vs"], scales if c["kind"] in TOP else None)
    if c["op"] == "write":
        s["Lx"] = lr.Layout(f"({d},{h},{c['tokens']}):(1,{d},{h * d})")
        return
    s["Lq"] = lr.Layout(f"({d},{h},{c['batch']}):(1,{d},{h * d})")
    width = s["table"].shape[1]
    if c["op"] == "prefix":
        plan = lr.prefix_attention_plan(s["Lq"], s["cache"], s["Lq"], s["prefix"].numel(), width, s["q"].dtype)
    elif c["op"] == "attend":
        plan = lr.block_attention_plan(s["Lq"], s["cache"], s["Lq"], c["count"], s["q"].dtype)
    else:
        s["Lk"] = lr.Layout(f"({d},{c['kv']},{pages}):(1,{d},{c['kv'] * d})")
        plan = lr.block_select_plan(s["Lq"], s["Lk"], width)
    s["workspace"] = torch.empty(plan["workspace_bytes"], dtype=torch.uint8, device=s["device"])


# ---------------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "axes":
        b, n, h, d = state["x"].shape
        y = _rotate(state["x"].float().view(b * n, h, d), state["positions"], c, -1 if c["backward"] else 1)
        y = y.to(state["x"].dtype).view(b, n, h, d)
        return {"y": y.transpose(1, 2).contiguous() if c["split"] else y}
    if c["op"] == "write":
        _put(c, state["ck"], state["ks"], _rotate(state["k"].float(), state["positions"], c, 1), state["slots"])
        _put(c, state["cv"], state["vs"], state["v"].float(), state["slots"])
        return _stored(state)
    if c["op"] == "prefix":
        return _attend_prefix(c, state)
    if c["op"] == "choose":
        return _choose(c, state)
    return _attend_blocks(c, state)


def _own(c, s):
    lr = s["lr"]
    if c["op"] == "axes":
        lr.rope_axes(s["x"], s["Lx"], s["y"], s["Ly"], s["positions"], s["rope"], pairs=c["pairs"], backward=c["backward"])
        return {"y": s["y"]}
    if c["op"] == "write":
        lr.cache_write_axes(s["cache"], s["k"], s["Lx"], s["v"], s["Lx"], s["slots"], s["rope"], s["positions"],
                            pairs=c["pairs"])
        return _stored(s)
    if c["op"] == "choose":
        lr.block_keys(s["cache"], s["slots"], s["keys"], s["Lk"])
        lr.block_select(s["q"], s["Lq"], s["keys"], s["Lk"], s["table"], s["lens"], c["page"], s["blocks"], first=c["first"],
                        last=c["last"], workspace=s["workspace"])
        return {"keys": s["keys"], "blocks": s["blocks"]}
    if c["op"] == "prefix":
        lr.prefix_attention(s["q"], s["Lq"], s["cache"], s["prefix"], s["prefix_len"], s["table"], s["lens"], s["out"], s["Lq"],
                            lse=s["lse"], workspace=s["workspace"])
    else:
        lr.block_attention(s["q"], s["Lq"], s["cache"], s["blocks"], s["table"], s["lens"], s["out"], s["Lq"], lse=s["lse"],
                           workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _stored(s):
    return {"k": s["ck"], "v": s["cv"], "ks": s["ks"], "vs": s["vs"]}


def _rotate(x, positions, c, sign):
    """x (tokens, heads, dim) in 32 bits, turned by its positions (axes, tokens); angles in 64 bits."""
    axis, f = _frequencies(c, x.device)
    a = positions[axis].double().t() * f
    cos, sin = a.cos().float().unsqueeze(-2), (sign * a.sin()).float().unsqueeze(-2)
    rot, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["pairs"] == "half":
        u, v = rot[..., :c["rot"] // 2], rot[..., c["rot"] // 2:]
        return torch.cat([u * cos - v * sin, v * cos + u * sin, rest], -1)
    u, v = rot[..., 0::2], rot[..., 1::2]
    return torch.cat([torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2), rest], -1)


def _page_first(c, x):
    """A cache tensor or its scales as (pages, slots, heads, ...)."""
    return x if c["layout"] == "tokens" else x.transpose(1, 2)


def _put(c, cache, scales, x, slots):
    if c["pad"]:  # a row without a slot repeats the first that has one
        keep = slots >= 0
        at = torch.where(keep, torch.arange(keep.numel(), device=slots.device), keep.int().argmax())
        slots, x = slots[at], x[at]
    page, slot = slots // c["page"], slots % c["page"]
    if c["kind"] not in TOP:
        _page_first(c, cache)[page, slot] = x.to(cache.dtype)
        return
    scale = (x.abs().amax(-1) / TOP[c["kind"]]).clamp(min=2.0 ** -126)
    code = (x.double() / scale.double().unsqueeze(-1)).clamp(-TOP[c["kind"]], TOP[c["kind"]])  # 64 bits: ties
    _page_first(c, cache.view(torch.uint8))[page, slot] = code.float().to(torch.float8_e4m3fn).view(torch.uint8)
    _page_first(c, scales)[page, slot] = scale


def _rows(c, s, which, page, slot):
    """Keys ("k") or values ("v") of slots as 32 bits, (..., heads, dim)."""
    cache, scales = s["c" + which], s[which + "s"]
    if c["kind"] == "e4m3":
        x = _page_first(c, cache.view(torch.uint8))[page, slot].view(torch.float8_e4m3fn).float()
    else:
        x = _page_first(c, cache)[page, slot].float()
    return x if scales is None else x * _page_first(c, scales)[page, slot].unsqueeze(-1)


def _attend_prefix(c, s):
    b, h, kv, d = c["batch"], c["heads"], c["kv"], c["dim"]
    g = h // kv
    q = s["q"].float().view(b, kv, g, d) / math.sqrt(d)
    t = torch.arange(s["prefix"].numel() * c["page"], device=s["device"])
    page, slot = s["prefix"].long()[t // c["page"]], t % c["page"]
    seen = t < s["prefix_len"]
    k, v = _rows(c, s, "k", page, slot), _rows(c, s, "v", page, slot)  # (t, kv, d)
    v = torch.where(seen[:, None, None], v, torch.zeros_like(v))
    rows = q.permute(1, 0, 2, 3).reshape(kv, b * g, d)
    one = torch.matmul(rows, k.permute(1, 2, 0).contiguous()).masked_fill(~seen, -math.inf)  # (kv, b g, t)
    u = torch.arange(s["table"].shape[1] * c["page"], device=s["device"])
    page, slot = s["table"].long()[:, u // c["page"]], (u % c["page"]).expand(b, -1)
    mine = u < s["lens"].unsqueeze(1)
    ko, vo = _rows(c, s, "k", page, slot), _rows(c, s, "v", page, slot)  # (b, u, kv, d)
    vo = torch.where(mine[:, :, None, None], vo, torch.zeros_like(vo))
    two = torch.matmul(q, ko.permute(0, 2, 3, 1).contiguous()).masked_fill(~mine[:, None, None, :], -math.inf)
    two = two.transpose(0, 1).reshape(kv, b * g, -1)
    top = torch.maximum(one.amax(-1, keepdim=True), two.amax(-1, keepdim=True)).clamp(min=-1e30)
    one, two = (one - top).exp(), (two - top).exp()
    total = one.sum(-1, keepdim=True) + two.sum(-1, keepdim=True)
    own_part = torch.matmul(two.view(kv, b, g, -1).transpose(0, 1).contiguous(), vo.transpose(1, 2).contiguous())
    o = (torch.matmul(one, v.transpose(0, 1).contiguous()).view(kv, b, g, d) + own_part.transpose(0, 1))
    o = o / total.clamp(min=1e-30).view(kv, b, g, 1)
    lse = (total.log() + top).view(kv, b, g)
    return {"out": o.transpose(0, 1).reshape(b, h, d).to(s["q"].dtype), "lse": lse.transpose(0, 1).reshape(b, h)}


def _mean(c, s, page, count):
    """The mean of the first `count` keys of pages, in 64 bits, (..., kv, dim)."""
    slot = torch.arange(c["page"], device=s["device"])
    k = _rows(c, s, "k", page.unsqueeze(-1).expand(*page.shape, c["page"]), slot.expand(*page.shape, c["page"]))
    k = torch.where((slot < count.unsqueeze(-1))[..., None, None], k, torch.zeros_like(k))
    return k.sum(-3, dtype=torch.float64) / count.clamp(min=1)[..., None, None]


def _choose(c, s):
    b, h, kv, d, p = c["batch"], c["heads"], c["kv"], c["dim"], c["page"]
    n, table, keys = s["lens"].long().unsqueeze(1), s["table"].long(), s["keys"]
    j = torch.arange(table.shape[1], device=s["device"])
    if c["new"]:  # every block of every sequence
        count = (n - j * p).clamp(min=0, max=p)
        page = torch.where(count > 0, table, s["spare"])
        keys[page] = torch.where((count > 0)[..., None, None], _mean(c, s, page, count).to(keys.dtype), keys[s["spare"]])
    else:  # the one that the new token lies in
        page, count = s["slots"] // p, s["slots"] % p + 1
        keys[page] = _mean(c, s, page, count).to(keys.dtype)
    # scores in 64 bits: which blocks are chosen hangs on values next to a border
    k = keys[table].double()  # (b, blocks, kv, d)
    q = s["q"].double().view(b, kv, h // kv, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()).amax(2)  # (b, kv, blocks)
    blocks = ((n + p - 1) // p)[:, None, :]
    kept = (j < c["first"]) | (j >= blocks - c["last"])
    score = score.masked_fill(kept, math.inf).masked_fill(j >= blocks, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :c["count"]]
    width = table.shape[1]
    order = torch.where(order < blocks, order, width).sort(-1).values
    out = s["blocks"]
    out.fill_(-1)
    out[..., :order.shape[-1]] = torch.where(order == width, -1, order).int()
    return {"keys": keys, "blocks": out}


def _attend_blocks(c, s):
    b, h, kv, d, p = c["batch"], c["heads"], c["kv"], c["dim"], c["page"]
    block = s["blocks"].long()  # (b, kv, count)
    slot = torch.arange(p, device=s["device"])
    page = s["table"].long().unsqueeze(1).expand(-1, kv, -1).gather(2, block.clamp(min=0))
    seen = (block.unsqueeze(-1) >= 0) & (block.unsqueeze(-1) * p + slot < s["lens"].long().view(b, 1, 1, 1))
    seen = seen.view(b, kv, 1, -1)
    head = torch.arange(kv, device=s["device"]).view(1, kv, 1, 1)
    k, v = (_head_rows(c, s, w, page.unsqueeze(-1), slot.view(1, 1, 1, p), head).view(b, kv, -1, d) for w in ("k", "v"))
    q = s["q"].float().view(b, kv, h // kv, d) / math.sqrt(d)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()).masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    w = (scores - top).exp()
    total = w.sum(-1, keepdim=True)
    v = torch.where(seen.transpose(2, 3), v, torch.zeros_like(v))
    o = torch.matmul(w, v) / total.clamp(min=1e-30)
    return {"out": o.reshape(b, h, d).to(s["q"].dtype), "lse": (total.log() + top).reshape(b, h)}


def _head_rows(c, s, which, page, slot, head):
    """Keys or values of one cache head each as 32 bits."""
    cache, scales = s["c" + which], s[which + "s"]
    if c["kind"] == "e4m3":
        x = _page_first(c, cache.view(torch.uint8))[page, slot, head].view(torch.float8_e4m3fn).float()
    else:
        x = _page_first(c, cache)[page, slot, head].float()
    return x if scales is None else x * _page_first(c, scales)[page, slot, head].unsqueeze(-1)


# ---------------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    e = BYTES[c["type"]]
    h, d = c["heads"], c["dim"]
    if c["op"] == "axes":
        tokens = c["batch"] * c["seq"]
        return {"bytes": 2 * tokens * h * d * e + 8 * c["axes"] * tokens, "flops": 3 * tokens * h * c["rot"]}
    row = d * BYTES[c["kind"]] + (4 if c["kind"] in TOP else 0)
    if c["op"] == "write":
        n = c["tokens"]
        return {"bytes": 2 * n * h * (d * e + row) + 8 * (c["axes"] + 1) * n, "flops": 4 * 2 * n * h * d}
    lens, p, kv = _lens(c), c["page"], c["kv"]
    io = c["batch"] * h * (2 * d * e + 4)  # queries, outputs and their log sums
    if c["op"] == "prefix":
        n = c["prefix"] + sum(lens)
        return {"bytes": 2 * n * kv * row + io + 4 * n // p, "flops": 4 * (c["prefix"] * c["batch"] + sum(lens)) * h * d}
    blocks = [-(-n // p) for n in lens]
    if c["op"] == "choose":
        new = sum(lens) if c["new"] else sum((n - 1) % p + 1 for n in lens)
        made = sum(blocks) if c["new"] else c["batch"]
        moved = new * kv * row + made * kv * d * e + sum(blocks) * (kv * d * e + 4) + c["batch"] * h * d * e
        return {"bytes": moved + 4 * c["batch"] * kv * c["count"], "flops": new * kv * d + 2 * sum(blocks) * h * d}
    tokens = sum(min(n, (c["count"] - 1) * p + (n - 1) % p + 1) for n in lens)
    return {"bytes": 2 * tokens * kv * row + io + 8 * c["batch"] * kv * c["count"], "flops": 4 * tokens * h * d}


# ---------------------------------------------------------------------------------- 64 bits
def _turned(x, positions, c, sign):
    """x (tokens, heads, dim) turned in complex numbers of 64 bits, an axis at a time."""
    rot, axes, sections = c["rot"], c["axes"], _sections(c)
    y = x.double().clone()
    for a in range(axes):
        if c["order"] == "blocks":
            pair = list(range(sum(sections[:a]), sum(sections[:a + 1])))
        else:
            pair = [i for i in range(a, rot // 2, axes) if a == 0 or i < axes * sections[a]]
            if a == 0:
                pair = sorted(pair + [i for i in range(rot // 2) if i % axes and i >= axes * sections[i % axes]])
        at = torch.tensor(pair, device=x.device)
        turn = torch.arange(len(pair), device=x.device).double() / len(pair) if c["own"] else at.double() * 2 / rot
        w = torch.exp(1j * sign * positions[a].double()[:, None] * torch.exp(-math.log(BASE) * turn))[:, None, :]
        i, k = (at, at + rot // 2) if c["pairs"] == "half" else (2 * at, 2 * at + 1)
        z = torch.complex(y[..., i], y[..., k]) * w
        y[..., i], y[..., k] = z.real, z.imag
    return y


def _nearest(x):
    """x rounded to the values that an e4m3 code stands for, ties to even."""
    x = x.clamp(-TOP["e4m3"], TOP["e4m3"])
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (x / step).round() * step


def _exact_rows(c, s, which, slots):
    """Keys or values of slots (n,) as 64 bits, (n, heads, dim)."""
    cache, scales, p = s["c" + which], s[which + "s"], c["page"]
    page, slot = torch.div(slots, p, rounding_mode="floor"), slots % p
    x = cache.view(torch.uint8) if c["kind"] == "e4m3" else cache
    x = x[page, slot] if c["layout"] == "tokens" else x[page, :, slot]
    x = (x.view(TYPES["e4m3"]).float() if c["kind"] == "e4m3" else x).double()
    if scales is None:
        return x
    return x * (scales[page, slot] if c["layout"] == "tokens" else scales[page, :, slot]).double()[..., None]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "axes":
        b, n, h, d = s["x"].shape
        y = torch.empty((b, h, n, d) if c["split"] else (b, n, h, d), dtype=torch.float64, device=s["device"])
        for i in range(b):
            z = _turned(s["x"][i], s["positions"][:, i * n:(i + 1) * n], c, -1 if c["backward"] else 1)
            y[i] = z.permute(1, 0, 2) if c["split"] else z
        return {"y": y}
    if c["op"] == "write":
        return _exact_store(c, s)
    if c["op"] == "prefix":
        return _exact_prefix(c, s)
    if c["op"] == "choose":
        return _exact_choice(c, s)
    b, h, kv, d, p = c["batch"], c["heads"], c["kv"], c["dim"], c["page"]
    out = torch.zeros((b, h, d), dtype=torch.float64, device=s["device"])
    lse = torch.full((b, h), -math.inf, dtype=torch.float64, device=s["device"])
    for i, n in enumerate(_lens(c)):
        blocks = s["blocks"][i].long()
        blocks = blocks[:, blocks[0] >= 0]  # as many for each head
        t = (blocks[..., None] * p + torch.arange(p, device=s["device"])).flatten(1)
        t = t[t < n].view(kv, -1)  # the last block is chosen for each head, and ends with the sequence
        slots = s["table"][i].long()[t // p] * p + t % p
        k, v = (torch.stack([_exact_rows(c, s, w, slots[g])[:, g] for g in range(kv)]) for w in ("k", "v"))
        q = s["q"][i].double().view(kv, h // kv, d)
        score = torch.matmul(k, (q * d ** -0.5).permute(0, 2, 1).contiguous())  # (kv, t, group)
        lse[i] = torch.logsumexp(score, 1).reshape(h)
        out[i] = torch.matmul(torch.softmax(score, 1).permute(0, 2, 1).contiguous(), v).reshape(h, d)
    return {"out": out, "lse": lse}


def _exact_store(c, s):
    out = {}
    for name, x, cache in (("k", s["k"], s["ck"]), ("v", s["v"], s["cv"])):
        x = _turned(x, s["positions"], c, 1) if name == "k" else x.double()
        p, h, d = c["page"], c["heads"], c["dim"]
        flat = torch.zeros((cache.shape[0] * p, h, d), dtype=torch.float64, device=s["device"])
        scales, keep = torch.zeros(flat.shape[:2], dtype=torch.float64, device=s["device"]), s["slots"] >= 0
        if c["kind"] in TOP:
            scale = x.abs().amax(-1) / TOP[c["kind"]]
            x = _nearest(x / scale[..., None])
            scales[s["slots"][keep]] = scale[keep]
        flat[s["slots"][keep]] = x[keep]
        flat, scales = flat.view(-1, p, h, d), scales.view(-1, p, h)
        if c["layout"] == "heads":
            flat, scales = flat.transpose(1, 2), scales.transpose(1, 2)
        out[name] = flat
        out[name + "s"] = scales if c["kind"] in TOP else None
    return out


def _exact_prefix(c, s):
    b, h, kv, d, p = c["batch"], c["heads"], c["kv"], c["dim"], c["page"]
    t = torch.arange(c["prefix"], device=s["device"])
    slots = s["prefix"].long()[t // p] * p + t % p
    kp, vp = (_exact_rows(c, s, w, slots).permute(1, 0, 2).contiguous() for w in ("k", "v"))  # (kv, t, d)
    out = torch.empty((b, h, d), dtype=torch.float64, device=s["device"])
    lse = torch.empty((b, h), dtype=torch.float64, device=s["device"])
    for i, n in enumerate(_lens(c)):
        t = torch.arange(n, device=s["device"])
        slots = s["table"][i].long()[t // p] * p + t % p
        ko, vo = (_exact_rows(c, s, w, slots).permute(1, 0, 2).contiguous() for w in ("k", "v"))
        q = (s["q"][i].double().view(kv, h // kv, d) * d ** -0.5).permute(0, 2, 1).contiguous()
        score = torch.cat([torch.matmul(kp, q), torch.matmul(ko, q)], 1)  # (kv, t, group)
        lse[i] = torch.logsumexp(score, 1).reshape(h)
        w = torch.softmax(score, 1).permute(0, 2, 1)
        out[i] = (torch.matmul(w[..., :c["prefix"]].contiguous(), vp) + torch.matmul(w[..., c["prefix"]:].contiguous(), vo)
                  ).reshape(h, d)
    return {"out": out, "lse": lse}


def _exact_choice(c, s):
    """A sequence at a time; the chosen blocks follow from the keys as they are stored."""
    b, h, kv, d, p = c["batch"], c["heads"], c["kv"], c["dim"], c["page"]
    keys = s["keys"].double()
    blocks = torch.full((b, kv, c["count"]), -1, dtype=torch.int32, device=s["device"])
    for i, n in enumerate(_lens(c)):
        many = -(-n // p)
        page = s["table"][i, :many].long()
        for first in range(0 if c["new"] else many - 1, many, 2048):
            at = torch.arange(first, min(first + 2048, many), device=s["device"])
            t = (at[:, None] * p + torch.arange(p, device=s["device"])).flatten()
            x = _exact_rows(c, s, "k", page[t // p] * p + t % p).view(-1, p, kv, d)
            x = x * (t < n).view(-1, p, 1, 1)
            keys[page[at]] = x.sum(1) / (n - at * p).clamp(max=p).view(-1, 1, 1)
        stored = keys[page].to(s["q"].dtype).double().permute(1, 0, 2).contiguous()  # (kv, blocks, d)
        score = torch.matmul(stored, s["q"][i].double().view(kv, h // kv, d).permute(0, 2, 1).contiguous()).amax(-1)
        j = torch.arange(many, device=s["device"])
        score[:, (j < c["first"]) | (j >= many - c["last"])] = math.inf
        # the lowest index first among equal scores
        rank = torch.sort(-score, dim=-1, stable=True).indices[:, :c["count"]].sort(-1).values
        blocks[i, :, :rank.shape[1]] = rank.int()
    return {"keys": keys, "blocks": blocks}
