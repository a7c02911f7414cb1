"""The operators for long and many-sided contexts on the GPU against plain 64-bit forms computed here on the CPU.

Tolerances count roundings: storing a value in type T is off by at most half a step, HALF[T] relative
(or half the smallest subnormal), and every 32-bit operation by 2^-24 of its result.  The forms in 64 bits that the
attention of test_gpu_operators has are used here too.
"""

import math

import pytest

torch = pytest.importorskip("torch")
import layout_remapping_copy_amd as lr  # noqa: E402

from test_gpu_operators import (F64, HALF, T, TINY, TOP, U, attention64, attention_case, cache_strides, close, content,  # noqa: E402,F401
                                dev, make_cache, quantised64, rand, rope_tolerance, tight64)

pytestmark = pytest.mark.gpu


def ints(lo, hi, shape, seed):
    return torch.randint(lo, hi, shape, generator=torch.Generator().manual_seed(seed))


# ------------------------------------------------------------------------------------ positions with several axes
def rotate64(x, positions, table, pairs, sign=1):
    """x (tokens, heads, dim) in 64 bits, positions (axes, tokens); the angle from the table's fractions of a turn."""
    rot, turns, m = table.rot_dim, table.turns.cpu(), table.magnitude
    at = positions[table.axis.cpu().long()].t()                       # (tokens, pairs)
    frac = (at * turns).to(F64) / 2.0 ** 64                           # int64 product wraps: whole turns drop out
    a = (frac * 2 * math.pi)[:, None, :]
    c, s = m * torch.cos(a), sign * m * torch.sin(a)
    y = x.to(F64).clone()
    u, v = (slice(0, rot // 2), slice(rot // 2, rot)) if pairs == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    p, q = y[..., u].clone(), y[..., v].clone()
    y[..., u], y[..., v] = p * c - q * s, q * c + p * s
    size = torch.zeros_like(y)   # |p| + |q| of each rotated element: what its 32-bit error is relative to
    size[..., u] = size[..., v] = (p.abs() + q.abs()) * m
    return y, size


AXES = [  # type, tokens, heads, dim, sections, order, own, pairs, order of y
    ("bf16", 7, 3, 128, [16, 24, 24], "blocks", False, "half", None),
    ("bf16", 7, 3, 128, [24, 20, 20], "cyclic", False, "interleaved", None),
    ("fp16", 1, 1, 64, [16, 16], "blocks", True, "half", None),
    ("fp32", 65, 5, 80, [20, 20], "blocks", True, "interleaved", None),
    ("fp32", 65, 5, 80, [8, 4, 4], "cyclic", True, "interleaved", "heads"),
    ("bf16", 33, 2, 72, [6, 4, 4, 4], "cyclic", False, "half", None),
    ("fp16", 33, 2, 33, [3, 0, 5], "blocks", True, "half", None), ("fp32", 9, 4, 20, [3], "blocks", False, "half", None),
    ("fp16", 5, 2, 33, [4, 4, 3], "blocks", False, "interleaved", None), ("fp32", 1, 1, 2, [0, 1], "blocks", False, "half", None),
    ("bf16", 130, 40, 96, [16, 8, 8], "cyclic", False, "half", "heads"),
    ("bf16", 257, 4, 1024, [172, 170, 170], "cyclic", True, "half", "heads"),
    ("fp32", 1030, 1, 128, [32, 32], "blocks", True, "half", "heads"),
    ("bf16", 13, 3, 24, [2, 1, 1], "blocks", False, "half", "column"),
    ("fp32", 13, 3, 24, [2, 1, 1], "cyclic", False, "interleaved", "column"),
]


@pytest.mark.parametrize("dtype,n,h,d,sections,order,own,pairs,out", AXES)
def test_rope_axes(dev, dtype, n, h, d, sections, order, own, pairs, out):
    t, rot = T[dtype], 2 * sum(sections)
    x = rand((n, h, d), t, n + d)
    positions = ints(-1000, 1 << 20, (len(sections), n), 1)
    table = lr.rope_axes_table(rot, sections, order=order, own=own, base=500000.0, scaling="bands", factor=8.0,
                               original_len=8192, low=1.0, high=4.0, device=dev)
    sy = {None: (h * d, d, 1), "heads": (d, n * d, 1), "column": (1, n * d, n)}[out]
    for backward in (False, True):
        y = torch.full((n * h * d,), -7.0, dtype=t, device=dev)
        lr.rope_axes(x.to(dev), f"({d},{h},{n}):(1,{d},{h * d})", y, f"({d},{h},{n}):({sy[2]},{sy[1]},{sy[0]})",
                     positions.to(dev), table, pairs=pairs, backward=backward)
        want, size = rotate64(x, positions, table, pairs, -1 if backward else 1)
        close(y.cpu().as_strided((n, h, d), sy), want, rope_tolerance(want, size, t), backward)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 34)])
def test_rope_axes_of_equal_positions_is_rope(dev, dtype, d):
    """With the same position on each axis and shared frequencies the result is rope's, bit by bit."""
    n, h = 50, 3
    x = rand((n, h, d), T[dtype], 7).to(dev)
    L = f"({d},{h},{n}):(1,{d},{h * d})"
    at = ints(0, 1 << 40, (n,), 3).to(dev)
    third = d // 2 // 3
    axes = lr.rope_axes_table(d, [d // 2 - 2 * third, third, third], order="cyclic", device=dev)
    got = lr.rope_axes(x, L, torch.empty_like(x), L, at.expand(3, n).contiguous(), axes)
    assert torch.equal(got, lr.rope(x, L, torch.empty_like(x), L, at, lr.rope_table(d, device=dev)))


@pytest.mark.parametrize("aligned", [True, False])
def test_rope_axes_layout_of_positions(dev, aligned):
    """Positions that lie token by token, shared over a batch; padded rows, a part of the tokens, an offset buffer."""
    b, n, h, d = 3, 11, 4, 32
    row = d + (8 if aligned else 3)
    x = rand((b * n, h, d), torch.bfloat16, 5)
    xb = torch.full((b * n * h * row,), float("nan"), dtype=torch.bfloat16)
    xb.as_strided((b * n, h, d), (h * row, row, 1)).copy_(x)
    table = lr.rope_axes_table(16, [4, 2, 2], device=dev)
    pos = ints(0, 5000, (n, 3), 2)
    y = torch.full((b * h * n * row + 1,), -7.0, dtype=torch.bfloat16, device=dev)
    L = f"({d},{h},({n},{b})):(1,{row},({h * row},{n * h * row}))"
    used, off = 2 * n + 4, 0 if aligned else 1
    lr.rope_axes(xb.to(dev), L, y[off:], L, pos.to(dev), table, Lp=f"(({n},{b}),3):((3,0),1)", n=used)
    want, size = rotate64(x, pos.t().repeat(1, b), table, "half")
    got = y.cpu()[off:].as_strided((b * n, h, d), (h * row, row, 1))
    close(got[:used], want[:used], rope_tolerance(want, size, torch.bfloat16)[:used])
    assert (got[used:] == -7).all() and int((y == -7).sum()) == y.numel() - used * h * d


def test_rope_axes_far_positions(dev):
    pos = torch.tensor([[0, 1, -1, 10 ** 9, 2 ** 40 + 1, -2 ** 63], [2 ** 63 - 1, -5, 7, 131071, -10 ** 9, 2 ** 62]])
    x = rand((6, 2, 64), torch.float32, 3)
    table = lr.rope_axes_table(64, [16, 16], own=True, device=dev)
    L = "(64,2,6):(1,64,128)"
    y = lr.rope_axes(x.to(dev), L, torch.empty(x.shape, device=dev), L, pos.to(dev), table)
    want, size = rotate64(x, pos, table, "half")
    close(y, want, rope_tolerance(want, size, torch.float32))
    # the table against the formula: the second axis has the frequencies of a rotation of its 16 pairs
    a = 131071 * 10000.0 ** (-torch.arange(16, dtype=F64) / 16)
    p, q = x[3, 0, 16:32].to(F64), x[3, 0, 48:].to(F64)
    close(y[3, 0, 16:32], p * a.cos() - q * a.sin(), 1e-6 * (p.abs() + q.abs()))


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 30)])
def test_rope_axes_in_place(dev, dtype, d):
    x = rand((50, 3, d), T[dtype], 7).to(dev)
    L, pos = f"({d},3,50):(1,{d},{3 * d})", ints(0, 100, (2, 50), 1).to(dev)
    table = lr.rope_axes_table(d, [d // 4, d // 2 - d // 4], device=dev)
    y = lr.rope_axes(x, L, torch.empty_like(x), L, pos, table)
    lr.rope_axes(x, L, x, L, pos, table)
    assert torch.equal(x, y)


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
def test_rope_axes_gradient_by_differences(dev, pairs):
    """The loss sum(w y^2)/2 is quadratic in x, so its central difference along a direction is the gradient's
    product with it for any step; with the gradient R^T (w y) from the backward call."""
    n, h, d = 37, 3, 48
    x, w, e = (rand((n, h, d), torch.float32, s).to(dev) for s in (1, 2, 3))
    L, pos = f"({d},{h},{n}):(1,{d},{h * d})", ints(0, 4000, (3, n), 4).to(dev)
    table = lr.rope_axes_table(32, [6, 5, 5], order="cyclic", scaling="parts", factor=4.0, original_len=2048, device=dev)

    def forward(z):
        return lr.rope_axes(z, L, torch.empty_like(z), L, pos, table, pairs=pairs)
    y = forward(x)
    grad = lr.rope_axes(w * y, L, torch.empty_like(x), L, pos, table, pairs=pairs, backward=True)
    up, down = forward(x + e).double(), forward(x - e).double()
    got = ((w.double() * (up ** 2 - down ** 2)).sum() / 4).item()
    want = (grad.double() * e.double()).sum().item()
    terms = (w.double().abs() * (up ** 2 + down ** 2)).sum().item() / 4 + (grad.double() * e.double()).abs().sum().item()
    assert abs(got - want) <= 16 * U * terms


def test_rope_axes_of_no_axis(dev):
    """A pair whose entry is no axis turns by the first one's position; nothing is read elsewhere."""
    L, pos = "(16,1,4):(1,16,16)", ints(0, 50, (2, 4), 4)
    for d in (16, 18):                                                 # in chunks, and element by element
        x = rand((4, 1, d), torch.float32, 1)
        table = lr.rope_axes_table(16, [4, 4], device=dev)
        table.axis = torch.tensor([0, 1, 2, -1, 1 << 30, -2 ** 31, 1, 5], dtype=torch.int32, device=dev)
        L = f"({d},1,4):(1,{d},{d})"
        y = lr.rope_axes(x.to(dev), L, torch.empty((4, 1, d), device=dev), L, pos.to(dev), table)
        table.axis = torch.tensor([0, 1, 0, 0, 0, 0, 1, 0], dtype=torch.int32)
        want, size = rotate64(x, pos, table, "half")
        close(y, want, rope_tolerance(want, size, torch.float32))


# ------------------------------------------------------------------------------------ the cache
@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,kind,n,h,d,sections,order,page", [
    ("bf16", "e4m3", 70, 8, 128, [24, 20, 20], "cyclic", 16), ("fp16", "int8", 33, 2, 96, [16, 16], "blocks", 16),
    ("fp32", "fp32", 9, 3, 80, [4, 2, 2], "blocks", 5), ("bf16", "bf16", 40, 4, 64, [8, 8, 8, 8], "cyclic", 8),
    ("bf16", "e4m3", 20, 2, 33, [4, 4], "blocks", 16), ("fp16", "e4m3", 1000, 8, 256, [22, 21, 21], "cyclic", 64),
    ("bf16", "bf16", 1, 1, 2, [1], "blocks", 1)])
def test_cache_write_axes(dev, dtype, kind, n, h, d, sections, order, page, pairs):
    """The keys that are stored are rope_axes' in 64 bits, rounded once; values and padding as cache_write has them."""
    t, pages = T[dtype], -(-n // page) + 2
    k, v = rand((n, h, d), t, 1), rand((n, h, d), t, 2)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(3))[:n].clone()
    if n > 8:
        slots[3], slots[5] = -1, pages * page
    positions = ints(0, 100000, (len(sections), n), 4)
    table = lr.rope_axes_table(2 * sum(sections), sections, order=order, base=500000.0, device=dev)
    cache, info = make_cache(dev, kind, "tokens", pages, page, h, d, d)
    plain, _ = make_cache(dev, kind, "tokens", pages, page, h, d, d)
    L = f"({d},{h},{n}):(1,{d},{h * d})"
    lr.cache_write_axes(cache, k.to(dev), L, v.to(dev), L, slots.to(dev), table, positions.to(dev), pairs=pairs)
    lr.cache_write(plain, k.to(dev), L, v.to(dev), L, slots.to(dev))
    assert torch.equal(cache.v, plain.v) and (kind not in TOP or torch.equal(cache.v_scale, plain.v_scale))
    want, size = rotate64(k, positions, table, pairs)
    keep = (slots >= 0) & (slots < pages * page)
    got, scales = content(cache, info, d, "k")
    others = torch.ones(pages * page, dtype=torch.bool)
    others[slots[keep]] = False
    assert (got[others] == 0).all()
    if kind not in TOP:
        close(got[slots[keep]], want[keep], rope_tolerance(want, size, t)[keep])
        return
    # 32-bit rotation, then a scale 2^-24 off, then a code half a step off (of 8 steps an octave, or of 1)
    amax = want.abs().amax(-1)
    scale = scales[slots[keep]].to(F64)
    err = (8 * U * size).amax(-1)
    close(scale, (amax / TOP[kind])[keep], ((err + 2 * U * amax) / TOP[kind])[keep])
    step = 2.0 ** -4 * want[keep].abs() + 2.0 ** -10 * scale[..., None] if kind == "e4m3" else 0.5 * scale[..., None]
    close(got[slots[keep]].to(F64) * scale[..., None], want[keep], step * (1 + 2.0 ** -10) + 8 * U * size[keep])


# ------------------------------------------------------------------------------------ a shared prefix
def int32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def prefix_case(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, lens, **kw):
    """attention_case whose first sequence is the prefix: the cache, the prefix's pages, the others' table, the slots of
    the prefix and of each sequence, and the numbers."""
    cache, table, slots, sides = attention_case(dev, dtype, kind, heads, kv, dk, dv, page, order,
                                                [prefix] + [max(n, 0) for n in lens], **kw)
    return cache, table[0].contiguous(), table[1:].contiguous(), slots[0], slots[1:], sides


PREFIX = [  # type, kind, heads, kv, dk, dv, page, order, prefix, lens
    ("bf16", "bf16", 8, 2, 128, 128, 16, "tokens", 300, [1, 15, 0, 129]),
    ("bf16", "bf16", 32, 8, 128, 128, 16, "heads", 1000, [5, 0, 33, 200, 64]),
    ("fp16", "fp16", 8, 8, 64, 64, 16, "heads", 77, [1, 2, 31]),
    ("fp32", "fp32", 6, 3, 128, 128, 16, "tokens", 130, [1, 0, 65]),
    ("bf16", "e4m3", 32, 8, 128, 128, 64, "heads", 700, [1, 63, 64, 65, 300]),
    ("fp16", "int8", 20, 1, 80, 80, 32, "tokens", 500, [1, 40, 90]),
    ("fp32", "int8", 5, 1, 64, 64, 16, "tokens", 100, [3, 10]),
    ("bf16", "bf16", 16, 1, 192, 128, 16, "tokens", 257, [0, 64, 3]),
    ("bf16", "bf16", 48, 1, 256, 256, 16, "heads", 200, [31] * 5),
    ("fp16", "fp16", 7, 1, 72, 72, 8, "tokens", 333, [9] * 12),
    ("bf16", "bf16", 4, 2, 33, 17, 5, "tokens", 250, [1, 4, 5, 6]),
    ("bf16", "e4m3", 14, 2, 112, 112, 1, "tokens", 77, [1, 20]),
    ("fp32", "e4m3", 4, 2, 96, 80, 8, "heads", 33, [3, 100]),
    ("bf16", "bf16", 4, 4, 128, 128, 16, "column", 100, [20, 0]),
    ("bf16", "bf16", 8, 8, 32, 32, 128, "tokens", 2049, [300] * 40),
    ("bf16", "bf16", 64, 8, 128, 128, 16, "heads", 3000, [(37 * i) % 50 for i in range(24)]),
    ("fp16", "fp16", 64, 8, 128, 128, 16, "tokens", 1500, [(37 * i) % 50 for i in range(24)]),
    ("bf16", "int8", 64, 4, 128, 128, 16, "tokens", 1500, [(37 * i) % 50 for i in range(24)]),
    ("bf16", "bf16", 1, 1, 64, 64, 16, "tokens", 1, [0]),
    ("bf16", "bf16", 2, 1, 128, 128, 16, "tokens", 5000, [1]),
    ("bf16", "bf16", 10, 2, 160, 96, 16, "tokens", 333, [7] * 30),
    ("fp16", "e4m3", 32, 4, 96, 96, 32, "heads", 2000, [(13 * i) % 40 for i in range(24)]),
]


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,prefix,lens", PREFIX)
def test_prefix_attention(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, lens):
    t, b = T[dtype], len(lens)
    cache, first, table, shared, slots, (kn, vn) = prefix_case(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, lens)
    q = rand((b, heads, dk), t, 11)
    out = torch.full((b, heads, dv), -7.0, dtype=t, device=dev)
    lse = torch.full((b, heads), -7.0, device=dev)
    Lq, Lo = f"({dk},{heads},{b}):(1,{dk},{heads * dk})", f"({dv},{heads},{b}):(1,{dv},{heads * dv})"
    lr.prefix_attention(q.to(dev), Lq, cache, first.to(dev), int32([prefix], dev), table.to(dev), int32(lens, dev), out, Lo,
                        lse=lse)
    seen = [torch.cat([shared, u]) for u in slots]
    want, wlse, tol = attention64(q, [kn[u] for u in seen], [vn[u] for u in seen], dk ** -0.5, t, kind)
    close(out, want, tol, "out")
    close(lse, wlse, tol.lse, "lse")


@pytest.mark.parametrize("dtype,kind", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "e4m3")])
def test_prefix_attention_rows_and_lengths(dev, dtype, kind):
    """Rows without a sequence, an empty prefix, lengths past the tables, pages that are none, a part of the batch, a
    table and a prefix wider than needed."""
    t, heads, kv, d, page = T[dtype], 8, 2, 64, 16
    lens = [20, -1, 0, 50]
    cache, first, table, shared, slots, (kn, vn) = prefix_case(dev, dtype, kind, heads, kv, d, d, page, "tokens", 90, lens)
    b = len(lens)
    q = rand((b + 1, heads, d), t, 3)
    L = f"({d},{heads},{b + 1}):(1,{d},{heads * d})"
    for prefix, own in ((90, lens), (0, lens), (-5, [20, 0, 0, 50]), (33, [5, -2 ** 31, 1, 0])):
        out = torch.full((b + 1, heads, d), -7.0, dtype=t, device=dev)
        lse = torch.full((b, heads), -7.0, device=dev)
        lr.prefix_attention(q.to(dev), L, cache, first.to(dev), int32([prefix], dev), table.to(dev), int32(own, dev), out, L,
                            lse=lse)
        seen = [torch.cat([shared[:max(prefix, 0)], u[:n]]) if n >= 0 else u[:0] for u, n in zip(slots, own)]
        want, wlse, tol = attention64(q[:b], [kn[u] for u in seen], [vn[u] for u in seen], d ** -0.5, t, kind)
        close(out[:b], want, tol, (prefix, "out"))
        close(lse, wlse, tol.lse, (prefix, "lse"))
        assert (out[b] == -7).all()
    # lengths past what the tables have room for, and pages outside the cache, which are left out
    full = first[:6].clone()                                            # 90 tokens: 6 pages, of which 5 are full
    full[1], full[3] = -1, 1 << 30
    out, lse = torch.empty((b, heads, d), dtype=t, device=dev), torch.empty((b, heads), device=dev)
    L4 = f"({d},{heads},{b}):(1,{d},{heads * d})"
    lr.prefix_attention(q[:b].to(dev), L4, cache, full[:5].contiguous().to(dev), int32([2 ** 31 - 1], dev),
                        table[:, :1].contiguous().to(dev), int32([2 ** 31 - 1, -1, 0, 2 ** 31 - 1], dev), out, L4, lse=lse)
    keep = torch.cat([shared[i * page:(i + 1) * page] for i in (0, 2, 4)])
    seen = [torch.cat([keep, slots[0][:page]]), keep[:0], keep, torch.cat([keep, slots[3][:page]])]
    want, wlse, tol = attention64(q[:b], [kn[u] for u in seen], [vn[u] for u in seen], d ** -0.5, t, kind)
    close(out, want, tol, "past")
    close(lse, wlse, tol.lse, "past lse")


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,prefix,lens", [PREFIX[1], PREFIX[3], PREFIX[4], PREFIX[10], PREFIX[15]])
def test_prefix_attention_is_paged_attention(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, lens):
    """Over whole pages of a prefix the result is paged_attention's over tables that begin with them, within both's
    tolerances; and twice the same call gives the same bits."""
    t, b, prefix = T[dtype], len(lens), -(-prefix // page) * page
    cache, first, table, shared, slots, (kn, vn) = prefix_case(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, lens)
    q = rand((b, heads, dk), t, 11)
    Lq, Lo = f"({dk},{heads},{b}):(1,{dk},{heads * dk})", f"({dv},{heads},{b}):(1,{dv},{heads * dv})"
    n = prefix // page
    both = torch.cat([first[:n].expand(b, n), table], 1).contiguous()
    one, two, again = (torch.empty((b, heads, dv), dtype=t, device=dev) for _ in range(3))
    args = (q.to(dev), Lq, cache, first[:n].contiguous().to(dev), int32([prefix], dev), table.to(dev), int32(lens, dev))
    lr.prefix_attention(*args, one, Lo)
    lr.prefix_attention(*args, again, Lo)
    assert torch.equal(one, again)
    lr.paged_attention(q.to(dev), Lq, cache, both.to(dev), int32([prefix + max(m, 0) for m in lens], dev), two, Lo)
    seen = [torch.cat([shared, u]) for u in slots]
    want, _, tol = attention64(q, [kn[u] for u in seen], [vn[u] for u in seen], dk ** -0.5, t, kind)
    close(one, two.to(F64).cpu(), 2 * tol)


@pytest.mark.parametrize("dtype,kind", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "int8")])
@pytest.mark.parametrize("wide", [True, False])
def test_prefix_attention_strides(dev, dtype, kind, wide):
    """Queries and outputs with strides, offset buffers, padded cache rows; other elements stay as they were."""
    t, b, heads, kv, d, page = T[dtype], 9, 16, 2, 64, 16
    pad = 8 if wide else 3
    cache, first, table, shared, slots, (kn, vn) = prefix_case(dev, dtype, kind, heads, kv, d, d, page, "heads", 200,
                                                               [3 * i for i in range(b)], pad=pad)
    row = d + pad
    q = rand((b, heads, d), t, 5)
    flat = torch.full((heads * b * row + 1,), float("nan"), dtype=t)
    flat[1:].as_strided((b, heads, d), (row, b * row, 1)).copy_(q)
    out = torch.full((heads * b * row + 1,), -7.0, dtype=t, device=dev)
    L = f"({d},{heads},{b}):(1,{b * row},{row})"
    lr.prefix_attention(flat.to(dev)[1:], L, cache, first.to(dev), int32([200], dev), table.to(dev),
                        int32([3 * i for i in range(b)], dev), out[1:], L, scale=0.3)
    seen = [torch.cat([shared, u]) for u in slots]
    want, _, tol = attention64(q, [kn[u] for u in seen], [vn[u] for u in seen], 0.3, t, kind)
    close(out.cpu()[1:].as_strided((b, heads, d), (row, b * row, 1)), want, tol)
    assert int((out == -7).sum()) == out.numel() - b * heads * d


@pytest.mark.parametrize("dtype,kind,d", [("bf16", "bf16", 128), ("fp16", "fp16", 128), ("fp32", "fp32", 64), ("bf16", "e4m3", 128)])
def test_prefix_attention_large_scores(dev, dtype, kind, d):
    """Scores of some thousands on one side of the prefix's end only: the other side's weight is nothing."""
    t, heads, kv, page, b = T[dtype], 32, 2, 16, 6
    cache, first, table, shared, slots, (kn, vn) = prefix_case(dev, dtype, kind, heads, kv, d, d, page, "heads", 400, [30] * b)
    q = rand((b, heads, d), t, 5) * 4
    out, lse = torch.empty((b, heads, d), dtype=t, device=dev), torch.empty((b, heads), device=dev)
    L = f"({d},{heads},{b}):(1,{d},{heads * d})"
    lr.prefix_attention(q.to(dev), L, cache, first.to(dev), int32([400], dev), table.to(dev), int32([30] * b, dev), out, L,
                        scale=4.0, lse=lse)
    seen = [torch.cat([shared, u]) for u in slots]
    want, wlse, tol = attention64(q, [kn[u] for u in seen], [vn[u] for u in seen], 4.0, t, kind)
    close(out, want, tol)
    close(lse, wlse, tol.lse)


def put_rows(cache, which, order, page, kv, d, slots, rows):
    pages = cache.k.numel() // (page * kv * d)
    s, _ = cache_strides(order, kv, page, d)
    x = getattr(cache, which).as_strided((pages, page, kv, d), s)
    x[slots.to(x.device) // page, slots.to(x.device) % page] = rows.to(x.device)


@pytest.mark.parametrize("dtype,heads", [("bf16", 32), ("fp16", 32), ("fp32", 32), ("bf16", 3)])
def test_prefix_attention_special_values(dev, dtype, heads):
    """An infinite value of the prefix makes its element infinite in every row, a NaN query its own rows NaN."""
    t, kv, d, page, b = T[dtype], 1, 128, 16, 5
    cache, first, table, shared, slots, (kn, vn) = prefix_case(dev, dtype, dtype, heads, kv, d, d, page, "tokens", 150, [9] * b)
    rows = vn[shared[77:78]].clone()
    rows[0, 0, 3], rows[0, 0, 64] = math.inf, -math.inf
    put_rows(cache, "v", "tokens", page, kv, d, shared[77:78], rows.to(t))
    q = rand((b, heads, d), t, 5)
    q[2, 1, 5] = math.nan
    out, lse = torch.empty((b, heads, d), dtype=t, device=dev), torch.empty((b, heads), device=dev)
    L = f"({d},{heads},{b}):(1,{d},{heads * d})"
    lr.prefix_attention(q.to(dev), L, cache, first.to(dev), int32([150], dev), table.to(dev), int32([9] * b, dev), out, L, lse=lse)
    out, lse = out.cpu(), lse.cpu()
    seen = [torch.cat([shared, u]) for u in slots]
    clean = torch.where(q.isnan(), torch.zeros_like(q), q)
    want, wlse, tol = attention64(clean, [kn[u] for u in seen], [vn[u] for u in seen], d ** -0.5, t, dtype)
    want[..., 3], want[..., 64] = math.inf, -math.inf
    want[2, 1], wlse[2, 1] = math.nan, math.nan
    close(out, want, tol)
    close(lse, wlse, tol.lse)


# Calls of enough rows and tokens to share tiles in shared memory: from 64 rows of a cache head on, 600000 rows times
# tokens (2^20 over 8-bit caches) that the prefix's pages have room for, 16-bit types, heads of up to 128.
ROWS = [  # type, kind, heads, kv, dk, dv, page, order, prefix, sequences, pages of the prefix's table
    ("bf16", "bf16", 16, 1, 128, 128, 16, "tokens", 3201, 12, 201), ("fp16", "fp16", 16, 1, 128, 128, 16, "heads", 4700, 8, 294),
    ("bf16", "bf16", 8, 2, 64, 64, 8, "tokens", 777, 32, 700), ("fp16", "fp16", 8, 2, 96, 80, 32, "heads", 500, 40, 150),
    ("bf16", "bf16", 5, 1, 72, 128, 5, "tokens", 333, 13, 2000), ("bf16", "bf16", 7, 1, 112, 40, 1, "heads", 130, 10, 9000),
    ("bf16", "e4m3", 16, 1, 128, 128, 64, "heads", 3300, 21, 52), ("fp16", "int8", 16, 1, 96, 96, 16, "tokens", 2800, 24, 176),
    ("bf16", "int8", 8, 1, 72, 64, 16, "heads", 1000, 24, 400), ("fp16", "e4m3", 8, 1, 128, 24, 16, "tokens", 90, 10, 900),
    ("bf16", "e4m3", 4, 4, 80, 128, 8, "tokens", 300, 70, 2000), ("fp16", "fp16", 4, 4, 8, 8, 16, "tokens", 64, 129, 400),
    ("bf16", "bf16", 16, 1, 32, 32, 16, "tokens", 40000, 4, 2500), ("bf16", "bf16", 1, 1, 128, 128, 16, "heads", 1, 64, 600),
    ("bf16", "bf16", 4, 1, 64, 128, 16, "tokens", 400, 500, 26), ("fp16", "e4m3", 1, 1, 128, 128, 16, "heads", 5000, 257, 313),
]


def rows_case(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, b, width, **kw):
    lens = [(37 * i) % 41 for i in range(b)]
    cache, first, table, shared, slots, sides = prefix_case(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, lens, **kw)
    wide = torch.full((max(width, -(-prefix // page)),), -1, dtype=torch.int32)
    wide[:-(-prefix // page)] = first[:-(-prefix // page)]
    return lens, cache, wide, table, shared, slots, sides


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,prefix,b,width", ROWS)
def test_prefix_attention_rows(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, b, width):
    t = T[dtype]
    assert b * heads // kv >= 64 and b * heads // kv * width * page >= (1 << 20 if kind in TOP else 600000)
    lens, cache, wide, table, shared, slots, (kn, vn) = rows_case(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, b, width)
    q = rand((b, heads, dk), t, 11)
    out, lse = torch.full((b, heads, dv), -7.0, dtype=t, device=dev), torch.full((b, heads), -7.0, device=dev)
    Lq, Lo = f"({dk},{heads},{b}):(1,{dk},{heads * dk})", f"({dv},{heads},{b}):(1,{dv},{heads * dv})"
    args = (q.to(dev), Lq, cache, wide.to(dev), int32([prefix], dev), table.to(dev), int32(lens, dev))
    lr.prefix_attention(*args, out, Lo, lse=lse)
    again = torch.empty_like(out)
    lr.prefix_attention(*args, again, Lo)
    assert torch.equal(out, again)
    some = list(range(0, b, max(1, b // 12))) + [b - 1]                 # the 64-bit form takes a sequence at a time
    seen = [torch.cat([shared, slots[i]]) for i in some]
    want, wlse, tol = attention64(q[some], [kn[u] for u in seen], [vn[u] for u in seen], dk ** -0.5, t, kind)
    close(out.cpu()[some], want, tol, "out")
    close(lse.cpu()[some], wlse, tol.lse, "lse")


@pytest.mark.parametrize("scale", [4.0, -0.7, 0.0])
@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,prefix,b,width", [ROWS[2], ROWS[3], ROWS[8], ROWS[9]])
def test_prefix_attention_rows_scales_and_pages(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, b, width, scale):
    """Large, negative and no scales; pages that are none inside the prefix; rows without a sequence; strided queries;
    a part of the batch, whose other rows stay."""
    t = T[dtype]
    lens, cache, wide, table, shared, slots, (kn, vn) = rows_case(dev, dtype, kind, heads, kv, dk, dv, page, order, prefix, b, width)
    wide[1], wide[2] = -1, 1 << 30
    kept = torch.cat([shared[:page], shared[3 * page:]])
    lens[1], lens[b - 2] = -1, -7
    row = dk + 3
    q = rand((b + 2, heads, dk), t, 11)
    flat = torch.full((heads * (b + 2) * row + 1,), float("nan"), dtype=t)
    flat[1:].as_strided(q.shape, (row, (b + 2) * row, 1)).copy_(q)
    out, lse = torch.full((b + 2, heads, dv), -7.0, dtype=t, device=dev), torch.full((b, heads), -7.0, device=dev)
    lr.prefix_attention(flat.to(dev)[1:], f"({dk},{heads},{b + 2}):(1,{(b + 2) * row},{row})", cache, wide.to(dev), int32([prefix], dev),
                        table.to(dev), int32(lens, dev), out, f"({dv},{heads},{b + 2}):(1,{dv},{heads * dv})", scale=scale, lse=lse)
    some = [0, 1, 2, b // 2, b - 2, b - 1]
    seen = [torch.cat([kept, slots[i]]) if lens[i] >= 0 else slots[i][:0] for i in some]
    want, wlse, tol = attention64(q[some], [kn[u] for u in seen], [vn[u] for u in seen], scale, t, kind)
    close(out.cpu()[some], want, tol, "out")
    close(lse.cpu()[some], wlse, tol.lse, "lse")
    assert (out[b:] == -7).all()


@pytest.mark.parametrize("dtype,kind", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3")])
def test_prefix_attention_rows_special_values(dev, dtype, kind):
    """Infinite values make their element infinite in every row, also where their weight has no second part; a NaN query
    its own rows NaN; what the cache holds in other slots (NaN) does not matter."""
    t, heads, kv, d, page, b, prefix = T[dtype], 8, 1, 64, 16, 20, 500
    lens, cache, wide, table, shared, slots, (kn, vn) = rows_case(dev, dtype, kind, heads, kv, d, d, page, "tokens", prefix, b, 500)
    q = rand((b, heads, d), t, 5)
    q[2, 1, 5] = math.nan
    if kind not in TOP:
        rows = vn[shared[77:78]].clone()
        rows[0, 0, 3], rows[0, 0, 40] = math.inf, -math.inf
        put_rows(cache, "v", "tokens", page, kv, d, shared[77:78], rows.to(t))
        put_rows(cache, "k", "tokens", page, kv, d, shared[77:78], torch.zeros(1, kv, d, dtype=t))
        kn[shared[77]] = 0                                              # its score is 0: a weight of one part at some base
    out, lse = torch.empty((b, heads, d), dtype=t, device=dev), torch.empty((b, heads), device=dev)
    L = f"({d},{heads},{b}):(1,{d},{heads * d})"
    lr.prefix_attention(q.to(dev), L, cache, wide.to(dev), int32([prefix], dev), table.to(dev), int32(lens, dev), out, L, lse=lse)
    seen = [torch.cat([shared, u]) for u in slots]
    clean = torch.where(q.isnan(), torch.zeros_like(q), q)
    want, wlse, tol = attention64(clean, [kn[u] for u in seen], [vn[u] for u in seen], d ** -0.5, t, kind)
    if kind not in TOP:
        want[..., 3], want[..., 40] = math.inf, -math.inf
    want[2, 1], wlse[2, 1] = math.nan, math.nan
    close(out.cpu(), want, tol)
    close(lse.cpu(), wlse, tol.lse)


@pytest.mark.parametrize("dtype,kind,weight,floor", [("bf16", "bf16", 2.0 ** -15, 0.0), ("fp16", "fp16", 2.0 ** -22, 2.0 ** -30),
                                                     ("fp16", "e4m3", 2.0 ** -15, 0.0)])
def test_prefix_attention_rows_weights_in_two_parts(dev, dtype, kind, weight, floor):
    """The weights have 16 bits (22 in fp16): values of one sign and size, whose sum one part of 8 bits would miss by more.
    A first part that is cut off leaves the second half a step of 2^-8 of what is below 2^-7: 2^-15 of the weight; fp16
    weights are kept from 0 by 2^-24 in the first part, which the second may not take off again, off a largest of 2^7."""
    t, heads, kv, d, page, b, prefix = T[dtype], 8, 1, 64, 16, 20, 700
    lens, cache, wide, table, shared, slots, (kn, vn) = rows_case(dev, dtype, kind, heads, kv, d, d, page, "heads", prefix, b, 500)
    q = rand((b, heads, d), t, 5)
    out = torch.empty((b, heads, d), dtype=t, device=dev)
    L = f"({d},{heads},{b}):(1,{d},{heads * d})"
    lr.prefix_attention(q.to(dev), L, cache, wide.to(dev), int32([prefix], dev), table.to(dev), int32([0] * b, dev), out, L)
    some = [0, 7, 19]
    want, tol = tight64(q[some], [kn[shared]] * 3, [vn[shared]] * 3, d ** -0.5, weight, floor)
    close(out.cpu()[some], want, tol)


@pytest.mark.parametrize("heads,kv,width", [(8, 1, 500), (32, 4, 2200)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_prefix_attention_rows_infinities(dev, dtype, heads, kv, width):
    """Infinite values at the ends of tiles, in places that different waves bring: their elements are infinite whatever the
    second part of their weights is, one of either sign and a NaN make NaN, and the others are as exact as ever."""
    t, d, page, b, prefix = T[dtype], 64, 16, 20, 300
    lens, cache, wide, table, shared, slots, (kn, vn) = rows_case(dev, dtype, dtype, heads, kv, d, d, page, "tokens", prefix, b, width)
    put = {0: (1, math.inf), 63: (2, -math.inf), 64: (3, math.inf), 95: (4, -math.inf), 200: (5, math.inf), 201: (5, -math.inf),
           256: (6, math.nan), 299: (63, math.inf)}
    clean = vn.clone()
    for at, (col, x) in put.items():
        vn[shared[at], :, col], clean[shared[at], :, col] = x, 0.0
    put_rows(cache, "v", "tokens", page, kv, d, shared, vn[shared].to(t))
    q = rand((b, heads, d), t, 5)
    out, lse = torch.empty((b, heads, d), dtype=t, device=dev), torch.empty((b, heads), device=dev)
    L = f"({d},{heads},{b}):(1,{d},{heads * d})"
    lr.prefix_attention(q.to(dev), L, cache, wide.to(dev), int32([prefix], dev), table.to(dev), int32(lens, dev), out, L, lse=lse)
    some = [0, 3, 11, b - 1]
    seen = [torch.cat([shared, slots[i]]) for i in some]
    want, wlse, tol = attention64(q[some], [kn[u] for u in seen], [clean[u] for u in seen], d ** -0.5, t, dtype)
    for col, x in ((1, math.inf), (2, -math.inf), (3, math.inf), (4, -math.inf), (5, math.nan), (6, math.nan), (63, math.inf)):
        want[..., col] = x
    close(out.cpu()[some], want, tol)
    close(lse.cpu()[some], wlse, tol.lse)


@pytest.mark.parametrize("heads,kv,width", [(8, 1, 500), (32, 4, 2200)])  # with the sequences' tokens in one launch, and alone
@pytest.mark.parametrize("dtype,kind,part", [("bf16", "bf16", 2.0 ** -19), ("fp16", "fp16", 2.0 ** -24),
                                             ("fp16", "e4m3", 2.0 ** -19), ("bf16", "int8", 2.0 ** -19)])
def test_prefix_attention_rows_two_tokens(dev, dtype, kind, part, heads, kv, width):
    """Two tokens of nearly equal weights and opposite values: what is left shows the weights' bits, which are the paged
    attention's.  The larger weight w is a power of two, the other w (1 - u) with u < 2^-10.  Its first part is w in bf16,
    and the second, below 2^-10 w, is off by half of its 2^-8: 2^-19 w; in fp16 the first is off by 2^-12 w and the second by
    2^-12 of that.  The output is half of these, rounded once; exponentials and sums in 32 bits are off by 2^-21 in all."""
    t, d, page, b = T[dtype], 64, 16, 20
    _, cache, wide, table, shared, _, _ = rows_case(dev, dtype, kind, heads, kv, d, d, page, "heads", 2, b, width)
    k = torch.zeros((2, kv, d), dtype=F64)
    k[0, :, 0], k[1, :, 0] = 1.0, 1 - 2.0 ** -8
    v = torch.ones((2, kv, d), dtype=F64)
    v[1] = -1
    if kind in TOP:                                                     # codes of 1 and -1, the difference in the scales
        pages = cache.k_scale.numel() // (page * kv)
        _, ss = cache_strides("heads", kv, page, d)
        at = shared.to(dev)
        for buf, sc, rows, scales in ((cache.k, cache.k_scale, (k != 0).float(), [1.0, 1 - 2.0 ** -8]),
                                      (cache.v, cache.v_scale, v.float(), [1.0, 1.0])):
            codes = rows.to(T[kind])
            s, _ = cache_strides("heads", kv, page, d)
            view = buf.as_strided((pages, page, kv, d), s)
            view[at // page, at % page] = (codes.view(torch.uint8) if kind == "e4m3" else codes).to(dev)
            sc.as_strided((pages, page, kv), ss)[at // page, at % page] = torch.tensor(scales, device=dev)[:, None].expand(2, kv)
    else:
        put_rows(cache, "k", "heads", page, kv, d, shared, k.to(t))
        put_rows(cache, "v", "heads", page, kv, d, shared, v.to(t))
    q = rand((b, heads, d), t, 11)
    q[..., 0] = (q[..., 0].abs() % 0.9375 + 0.0625).to(t)
    out, lse = torch.empty((b, heads, d), dtype=t, device=dev), torch.empty((b, heads), device=dev)
    L = f"({d},{heads},{b}):(1,{d},{heads * d})"
    lr.prefix_attention(q.to(dev), L, cache, wide.to(dev), int32([2], dev), table.to(dev), int32([0] * b, dev), out, L,
                        scale=0.25, lse=lse)
    u = q[..., 0].to(F64) * 0.25
    w = torch.exp(-u * 2.0 ** -8)
    want = ((1 - w) / (1 + w))[..., None].expand(b, heads, d)
    close(out, want, HALF[t] * want + part / 2 + 2.0 ** -21)
    close(lse, u + torch.log1p(w), 2.0 ** -21)


# ------------------------------------------------------------------------------------ blocks: their keys
KEYS = [  # type, kind, heads, d, page, order, lens
    ("bf16", "bf16", 8, 128, 16, "tokens", [100, 1, 16, 17]), ("bf16", "e4m3", 8, 128, 64, "heads", [300, 64, 1]),
    ("fp16", "int8", 2, 80, 32, "tokens", [70, 33]), ("fp32", "fp32", 3, 96, 8, "heads", [20, 8, 7]),
    ("fp32", "e4m3", 1, 256, 128, "tokens", [200]), ("bf16", "bf16", 2, 33, 5, "tokens", [23, 4, 5]),
    ("fp16", "fp16", 1, 512, 16, "tokens", [40]), ("bf16", "int8", 4, 72, 1, "tokens", [9]),
    ("bf16", "bf16", 2, 64, 16, "column", [50]), ("bf16", "e4m3", 3, 24, 16, "heads", [3000, 5]),
    ("fp16", "e4m3", 5, 300, 48, "tokens", [100]), ("bf16", "bf16", 16, 128, 16, "heads", [20000, 9000]),
]


@pytest.mark.parametrize("dtype,kind,h,d,page,order,lens", KEYS)
def test_block_keys(dev, dtype, kind, h, d, page, order, lens):
    """The keys after a prompt and after one more token a sequence, against means in 64 bits; other pages' keys stay."""
    t = T[dtype]
    grown = [n + 1 for n in lens]
    cache, table, slots, (kn, _) = attention_case(dev, dtype, kind, h, h, d, d, page, order, grown)
    pages = cache.k.numel() // (page * h * d)
    keys = torch.full((pages, h, d), -7.0, dtype=t, device=dev)
    L = f"({d},{h},{pages}):(1,{d},{h * d})"
    want = torch.full((pages, h, d), -7.0, dtype=F64)
    size = torch.zeros((pages, h, d), dtype=F64)

    def expect(i, n):                                                   # the blocks that sequence i's first n tokens lie in
        for j in range(-(-n // page)):
            rows = kn[slots[i][j * page:min(n, (j + 1) * page)]]
            want[table[i, j]], size[table[i, j]] = rows.mean(0), rows.abs().mean(0)
    prompt = torch.cat([u[:n] for u, n in zip(slots, lens)] + [torch.tensor([-1, pages * page, 2 ** 40])])
    lr.block_keys(cache, prompt.to(dev), keys, L)
    for i, n in enumerate(lens):
        expect(i, n)
    # sums in 64 bits, then two roundings
    close(keys, want, (HALF[t] * (1 + 2 * U) + U) * want.abs() + 2.0 ** -50 * size + TINY[t])
    step = torch.stack([u[-1] for u in slots])
    lr.block_keys(cache, step.to(dev), keys, L)
    for i, n in enumerate(grown):
        expect(i, n)
    close(keys, want, (HALF[t] * (1 + 2 * U) + U) * want.abs() + 2.0 ** -50 * size + TINY[t])
    assert lr.block_keys(cache, step[:0].to(dev), keys, L) is keys


def test_block_keys_layout(dev):
    """Keys with a layout of their own (pages next to each other), in another type than an 8-bit cache's queries."""
    h, d, page = 2, 64, 16
    cache, table, slots, (kn, _) = attention_case(dev, "bf16", "int8", h, h, d, d, page, "tokens", [40])
    pages = cache.k.numel() // (page * h * d)
    keys = torch.full((d * h * pages,), -7.0, device=dev)
    lr.block_keys(cache, slots[0].to(dev), keys, f"({d},{h},{pages}):({pages},{d * pages},1)")
    got = keys.cpu().as_strided((pages, h, d), (1, d * pages, pages))
    for j in range(3):
        rows = kn[slots[0][j * page:(j + 1) * page]]
        close(got[table[0, j]], rows.mean(0), 2 * U * rows.mean(0).abs() + 2.0 ** -50)
    assert int((keys == -7).sum()) == (pages - 3) * h * d


@pytest.mark.parametrize("dtype,tiny", [("bf16", 2.0 ** -36), ("fp16", 2.0 ** -24)])
@pytest.mark.parametrize("d", [24, 25])
def test_block_keys_are_rounded_twice(dev, dtype, tiny, d):
    """The mean is rounded to 32 bits and then to the type: a little off the middle of two numbers of the type, by what 32
    bits do not hold, it becomes that middle, and then the even one of the two."""
    t, page, eps = T[dtype], 16, torch.finfo(T[dtype]).eps
    k = torch.zeros((2 * page, 1, d), dtype=F64)
    k[0], k[page] = 16.0, -16.0
    k[3, 0, ::2], k[5, 0, ::2] = 8 * eps, tiny                          # 1 + eps / 2, and a little more
    k[page + 1, 0, ::2], k[page + 2, 0, ::2] = -24 * eps, tiny          # -1 - 3 eps / 2, and a little less
    assert torch.equal(k.to(t).to(F64), k)
    cache, _ = make_cache(dev, dtype, "tokens", 2, page, 1, d, d)
    L, slots = f"({d},1,{2 * page}):(1,{d},{d})", torch.arange(2 * page, device=dev)
    lr.cache_write(cache, k.to(t).to(dev), L, k.to(t).to(dev), L, slots)
    keys = lr.block_keys(cache, slots, torch.empty((2, 1, d), dtype=t, device=dev), f"({d},1,2):(1,{d},{d})").cpu()
    assert (keys[0] == 1).all() and (keys[1, 0, 1::2] == -1).all() and (keys[1, 0, ::2] == -1 - 2 * eps).all()
    assert torch.equal(keys, k.view(2, page, 1, d).mean(1).float().to(t))


@pytest.mark.parametrize("n", [9, 49, 103, 123])
@pytest.mark.parametrize("d", [64, 33])
def test_block_keys_between_two_numbers(dev, n, d):
    """Means just between two numbers of 32 bits become the even one: the sum is divided, as times 1 / n it would be off."""
    g = torch.Generator().manual_seed(n)
    q = torch.randint(1 << 24, 30 << 20, (d,), generator=g) | 1         # 25 bits, the last one set
    rows = torch.empty((128, 1, d), dtype=torch.int64)
    rows[n - 1] = (1 << 24) - 1                                         # the one odd number; the others even, of 24 bits
    left = n * q - rows[n - 1, 0]
    even = left // (2 * (n - 1)) * 2
    rows[:n - 1, 0] = even
    rows[:n - 1, 0] += 2 * (torch.arange(n - 1)[:, None] < ((left - (n - 1) * even) // 2)[None])
    rows[n:] = 5
    assert torch.equal(rows[:n, 0].sum(0), n * q) and torch.equal(rows.float().long(), rows)
    cache, _ = make_cache(dev, "fp32", "tokens", 1, 128, 1, d, d)
    L = f"({d},1,128):(1,{d},{d})"
    x = rows.float().to(dev)
    lr.cache_write(cache, x, L, x, L, torch.arange(128, device=dev))
    keys = lr.block_keys(cache, torch.arange(n, device=dev), torch.empty((1, 1, d), device=dev), f"({d},1,1):(1,{d},{d})")
    assert torch.equal(keys.cpu()[0, 0], q.to(F64).float())


@pytest.mark.parametrize("dtype,kind,h,d,page,lens,runs,total", [
    ("bf16", "bf16", 1, 32, 16, [100, 33, 16, 1], (0, 1), 0),           # an entry or none outside the cache behind each
    ("bf16", "e4m3", 2, 64, 16, [100, 60], (0, 70), 0),                 # more than a wave looks at
    ("fp16", "fp16", 8, 32, 64, [130, 70], (0, 6000), 0),               # many steps of looking on
    ("bf16", "bf16", 4, 32, 16, [9000], (0, 2), 0),                     # workgroups of several entries
    ("fp32", "fp32", 5, 20, 5, [4000, 333], (0, 1), 30000),             # a long end of padding
    ("bf16", "int8", 8, 32, 16, [60001, 20000], (0, 1), 140000),        # workgroups of 64 entries
])
def test_block_keys_of_padded_slots(dev, dtype, kind, h, d, page, lens, runs, total):
    """Slots outside the cache anywhere, also between those of one page and across the ends of workgroups: passed over."""
    t, g = T[dtype], torch.Generator().manual_seed(8)
    cache, table, slots, (kn, _) = attention_case(dev, dtype, kind, h, h, d, d, page, "tokens", lens)
    pages = cache.k.numel() // (page * h * d)
    numbers = kn.float().to(F64) if dtype != "fp32" else kn
    want = torch.full((pages, h, d), -7.0, dtype=t)
    for i, n in enumerate(lens):
        for j in range(-(-n // page)):
            want[int(table[i, j])] = numbers[slots[i][j * page:min(n, (j + 1) * page)]].mean(0).float().to(t)
    every = torch.cat(slots)
    holes = torch.randint(runs[0], runs[1] + 1, (every.numel(),), generator=g)
    if runs[1] > 100:                                                   # long runs here and there
        holes *= (torch.rand(every.numel(), generator=g) < 0.05)
    at = torch.arange(every.numel()) + holes.cumsum(0)
    padded = torch.full((max(total, int(at[-1]) + 1),), -1)
    padded[1::3], padded[2::7] = pages * page, -2 ** 63
    padded[at] = every
    keys = lr.block_keys(cache, padded.to(dev), torch.full((pages, h, d), -7.0, dtype=t, device=dev),
                         f"({d},{h},{pages}):(1,{d},{h * d})")
    assert torch.equal(keys.cpu(), want)
    rest = torch.full((pages, h, d), -7.0, dtype=t, device=dev)         # none inside the cache
    lr.block_keys(cache, torch.full((5000,), -1, device=dev), rest, f"({d},{h},{pages}):(1,{d},{h * d})")
    assert (rest == -7).all()


# ------------------------------------------------------------------------------------ blocks: the choice
def chosen64(q, keys, table, lens, page, count, first, last):
    """The choice by its definition: scores in 64 bits, sorted by (score, index)."""
    b, heads, d = q.shape
    pages, kv, _ = keys.shape
    out = torch.full((b, kv, count), -1, dtype=torch.int32)
    for i, n in enumerate(lens):
        many = min(-(-max(n, 0) // page), table.shape[1])
        for g in range(kv):
            if many <= count:
                out[i, g, :many] = torch.arange(many)
                continue
            at = table[i, :many].long()
            ok = (at >= 0) & (at < pages)
            k = keys[torch.where(ok, at, 0), g].to(F64)
            s = (k @ q[i, g * heads // kv:(g + 1) * heads // kv].to(F64).t())
            s = torch.where(s.isnan(), -math.inf, s).amax(-1)
            s = torch.where(ok, s, -math.inf).tolist()
            middle = sorted(range(first, many - last), key=lambda j: (-s[j], j))[:count - first - last]
            out[i, g] = torch.tensor(list(range(first)) + sorted(middle) + list(range(many - last, many)))
    return out


SELECT = [  # type, heads, kv, d, page, lens, count, first, last
    ("bf16", 32, 8, 128, 16, [4000, 1, 0, 300, 257], 16, 1, 2), ("fp16", 4, 4, 64, 64, [5000, 640, 641], 10, 0, 1),
    ("fp32", 6, 2, 96, 8, [1000, 37], 5, 1, 1), ("bf16", 40, 1, 256, 16, [3000], 40, 4, 4),
    ("bf16", 5, 1, 33, 5, [700, 2], 8, 0, 0), ("fp16", 7, 7, 72, 1, [900], 100, 10, 20), ("fp32", 1, 1, 20, 3, [500], 1, 0, 0),
    ("fp32", 3, 1, 130, 3, [500], 2, 1, 1), ("bf16", 66, 2, 128, 16, [2000], 12, 1, 1),
    ("bf16", 2, 1, 64, 1, [70000, 4097, 4096], 64, 1, 1), ("bf16", 16, 2, 128, 16, [40000] * 3, 2000, 1, 1),
    ("bf16", 8, 8, 128, 16, [17 * i for i in range(70)], 9, 1, 1),
]


@pytest.mark.parametrize("dtype,heads,kv,d,page,lens,count,first,last", SELECT)
@pytest.mark.parametrize("values", ["normal", "few"])
def test_block_select(dev, dtype, heads, kv, d, page, lens, count, first, last, values):
    """The choice is exact.  Keys of few values have many equal scores, of which the first are taken."""
    t, b = T[dtype], len(lens)
    width = max(-(-n // page) for n in lens) + 1
    pages = width * b + 2
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int()[:width * b].view(b, width)
    q, keys = rand((b, heads, d), t, 2), rand((pages, kv, d), t, 3)
    if values == "few":
        q, keys = ints(-1, 2, (b, heads, d), 2).to(t), torch.zeros((pages, kv, d), dtype=t)
        keys[..., 0] = ints(-2, 3, (pages, kv), 3).to(t)
    out = torch.full((b + 1, kv, count), -7, dtype=torch.int32, device=dev)
    Lq, Lk = f"({d},{heads},{b}):(1,{d},{heads * d})", f"({d},{kv},{pages}):(1,{d},{kv * d})"
    lr.block_select(q.to(dev), Lq, keys.to(dev), Lk, table.to(dev), int32(lens, dev), page, out, first=first, last=last)
    want = chosen64(q, keys, table, lens, page, count, first, last)
    assert torch.equal(out[:b].cpu(), want) and (out[b] == -7).all()


@pytest.mark.parametrize("dtype,kind,kv,d,page,order,lens", [("bf16", "e4m3", 4, 128, 16, "tokens", [20000, 16 * 999 + 3]),
                                                             ("fp16", "int8", 2, 80, 8, "heads", [8001, 8000]),
                                                             ("fp32", "e4m3", 2, 64, 16, "tokens", [16000])])
def test_block_keys_and_choice_bit_by_bit(dev, dtype, kind, kv, d, page, order, lens):
    """Keys of an 8-bit cache of thousands of pages equal, bit by bit, the 64-bit mean of the numbers that the cache gives in
    32 bits (of codes times scales for keys of 32 bits), rounded to 32 bits and then to the type; the choice is the one from
    those keys."""
    t, b, heads, count = T[dtype], len(lens), 4 * kv, 64
    cache, table, slots, (kn, _) = attention_case(dev, dtype, kind, heads, kv, d, d, page, order, lens)
    pages = cache.k.numel() // (page * kv * d)
    Lk, Lq = f"({d},{kv},{pages}):(1,{d},{kv * d})", f"({d},{heads},{b}):(1,{d},{heads * d})"
    every = torch.cat(slots)
    read, rest = (torch.empty((every.numel(), kv, d), dtype=torch.float32, device=dev) for _ in range(2))
    Lr = f"({d},{kv},{every.numel()}):(1,{d},{kv * d})"
    lr.cache_read(cache, every.to(dev), read, Lr, rest, Lr)
    assert torch.equal(read.cpu(), kn[every].float())                   # one rounding of code * scale
    numbers = kn if dtype == "fp32" else kn.float().to(F64)
    want = torch.zeros((pages, kv, d), dtype=t)
    for i, n in enumerate(lens):
        whole = n // page * page
        want[table[i, :n // page].long()] = numbers[slots[i][:whole]].view(-1, page, kv, d).mean(1).float().to(t)
        if n > whole:
            want[int(table[i, n // page])] = numbers[slots[i][whole:n]].mean(0).float().to(t)
    keys = lr.block_keys(cache, every.to(dev), torch.zeros((pages, kv, d), dtype=t, device=dev), Lk)
    assert torch.equal(keys.cpu(), want)
    q = rand((b, heads, d), t, 9)
    out = torch.empty((b, kv, count), dtype=torch.int32, device=dev)
    lr.block_select(q.to(dev), Lq, keys, Lk, table.to(dev), int32(lens, dev), page, out)
    assert torch.equal(out.cpu(), chosen64(q, want, table, lens, page, count, 1, 1))


def test_block_select_special_scores(dev):
    """Infinities, NaN, zeros of both signs, pages that are none, lengths past the table, strided and offset tensors."""
    b, heads, kv, d, page, width = 3, 4, 2, 32, 16, 40
    pages = 130
    table = torch.arange(b * width).int().view(b, width)
    table[0, 5], table[0, 6], table[1, 7], table[1, 0] = -1, pages, 1 << 30, -2 ** 31
    q, keys = rand((b, heads, d), torch.float32, 2), rand((pages, kv, d), torch.float32, 3)
    keys[3], keys[4, :, 2], keys[9], keys[10], keys[44, 0, 1], keys[45] = 0.0, math.inf, -0.0, 0.0, math.nan, -math.inf
    q[2, 0] = math.nan                                                  # the other head of its cache head decides
    q[1, 2:] = math.nan                                                 # no head does: all scores equal
    q[0, 1] = 0.0
    lens = [width * page, 2 ** 31 - 1, width * page - 3]
    row = d + 3
    qb, kb = torch.full((heads * b * row + 1,), math.nan), torch.full((kv * pages * row + 1,), math.nan)
    qb[1:].as_strided((b, heads, d), (row, b * row, 1)).copy_(q)
    kb[1:].as_strided((pages, kv, d), (row, pages * row, 1)).copy_(keys)
    for count, first, last in ((7, 1, 1), (7, 0, 0), (30, 3, 2), (39, 0, 0)):
        out = torch.full((b, kv, count), -7, dtype=torch.int32, device=dev)
        want = chosen64(q, keys, table, lens, page, count, first, last)
        lr.block_select(q.to(dev), f"({d},{heads},{b}):(1,{d},{heads * d})", keys.to(dev), f"({d},{kv},{pages}):(1,{d},{kv * d})",
                        table.to(dev), int32(lens, dev), page, out, first=first, last=last)
        assert torch.equal(out.cpu(), want), (count, first, last)
        lr.block_select(qb.to(dev)[1:], f"({d},{heads},{b}):(1,{b * row},{row})", kb.to(dev)[1:],
                        f"({d},{kv},{pages}):(1,{pages * row},{row})", table.to(dev), int32(lens, dev), page, out.fill_(-7),
                        first=first, last=last)
        assert torch.equal(out.cpu(), want), ("strided", count, first, last)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("queries,keys_as", [("column", "dense"), ("padded", "dense"), ("one", "dense"), ("dense", "padded"),
                                             ("dense", "column"), ("column", "padded"), ("wide", "wide")])
def test_block_select_strides(dev, dtype, queries, keys_as):
    """Queries and keys each with a layout of their own: dense, padded to whole chunks or by an odd count in an offset
    buffer, head dimensions apart, one number for a whole row; the choice is the dense ones'."""
    t, b, heads, kv, d, page, width = T[dtype], 3, 10, 2, 64, 16, 300
    lens, count = [width * page, 1234, 17], 20
    pages = b * width + 2
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).int()[:b * width].view(b, width)
    q, keys = rand((b, heads, d), t, 2), rand((pages, kv, d), t, 3)
    if queries == "one":
        q = q[..., :1].expand(b, heads, d).contiguous()

    def laid(x, how):                                                   # (buffer, offset, strides of d, heads, items)
        n, h, _ = x.shape
        if how == "one":
            return x[..., 0].contiguous(), 0, (0, 1, h)
        off, st = {"dense": (0, (1, d, h * d)), "padded": (1, (1, n * (d + 3), d + 3)), "wide": (8, (1, n * (d + 8), d + 8)),
                   "column": (0, (h, 1, h * d))}[how]
        buf = torch.full((off + n * h * (d + 8),), math.nan, dtype=t)
        buf[off:].as_strided((n, h, d), (st[2], st[1], st[0])).copy_(x)
        return buf, off, st
    qb, qo, qs = laid(q, queries)
    kb, ko, ks = laid(keys, keys_as)
    out = torch.full((b, kv, count), -7, dtype=torch.int32, device=dev)
    lr.block_select(qb.to(dev).view(-1)[qo:], f"({d},{heads},{b}):({qs[0]},{qs[1]},{qs[2]})", kb.to(dev)[ko:],
                    f"({d},{kv},{pages}):({ks[0]},{ks[1]},{ks[2]})", table.to(dev), int32(lens, dev), page, out)
    assert torch.equal(out.cpu(), chosen64(q, keys, table, lens, page, count, 1, 1))


def test_block_select_by_last_bits(dev):
    """Scores that differ in the 40th bit, and scores of every size: the border is found at any bit."""
    d, page, n = 32, 1, 3000
    g = torch.Generator().manual_seed(1)
    table = torch.randperm(n, generator=g).int().view(1, n)
    q = torch.zeros((1, 1, d))
    q[0, 0, :2] = torch.tensor([1.0, 2.0 ** -40])
    keys = torch.zeros((n, 1, d))
    keys[:, 0, 0], keys[:, 0, 1] = 1.0, torch.randperm(n, generator=g).float()
    huge = torch.zeros((n, 1, d))
    huge[:, 0, 0] = torch.randn(n, generator=g) * torch.exp2(torch.randint(-120, 120, (n,), generator=g).float())
    for k in (keys, huge):
        for count in (1, 2, 100, 1500, 2999):
            out = torch.empty((1, 1, count), dtype=torch.int32, device=dev)
            lr.block_select(q.to(dev), f"({d},1,1):(1,{d},{d})", k.to(dev), f"({d},1,{n}):(1,{d},{d})", table.to(dev), int32([n], dev),
                            page, out, first=0, last=0)
            assert torch.equal(out.cpu(), chosen64(q, k, table, [n], page, count, 0, 0)), count


# ------------------------------------------------------------------------------------ blocks: their attention
def blocks_seen(slots, blocks, n, page):
    """The slots of the tokens that a head's list of blocks holds, in the list's order."""
    many = -(-n // page)
    parts = [slots[j * page:min((j + 1) * page, n)] for j in blocks[:many].tolist() if 0 <= j < many]
    return torch.cat(parts) if parts else slots[:0]


def head_attention64(q, kn, vn, seen, kv, scale, t, kind):
    """attention64 of each (sequence, cache head) by itself; seen[i][g]: slots."""
    b, heads, dk = q.shape
    grp = heads // kv
    pairs = [(i, g) for i in range(b) for g in range(kv)]
    want, lse, tol = attention64(q.reshape(b * kv, grp, dk), [kn[seen[i][g]][:, g:g + 1] for i, g in pairs],
                                 [vn[seen[i][g]][:, g:g + 1] for i, g in pairs], scale, t, kind)
    out = tol.reshape(b, heads, -1)
    out.lse = tol.lse.reshape(b, heads)
    return want.reshape(b, heads, -1), lse.reshape(b, heads), out


BLOCKS = [  # type, kind, heads, kv, dk, dv, page, order, lens, count
    ("bf16", "bf16", 8, 2, 128, 128, 16, "tokens", [1, 15, 0, 129, 700], 5),
    ("bf16", "bf16", 32, 8, 128, 128, 64, "heads", [1000, 64, 65, 3000], 9),
    ("fp16", "fp16", 8, 8, 64, 64, 16, "heads", [31, 500], 40), ("fp32", "fp32", 6, 3, 128, 128, 16, "tokens", [0, 65, 300], 4),
    ("bf16", "e4m3", 32, 8, 128, 128, 64, "heads", [63, 1000, 64], 6), ("fp16", "int8", 20, 1, 80, 80, 32, "tokens", [40, 900], 11),
    ("fp32", "int8", 5, 1, 64, 64, 16, "tokens", [100], 3), ("bf16", "bf16", 16, 1, 192, 128, 16, "tokens", [257, 64], 7),
    ("bf16", "bf16", 48, 1, 256, 256, 16, "heads", [200, 31], 5), ("fp16", "fp16", 7, 1, 72, 72, 8, "tokens", [9, 333], 17),
    ("bf16", "bf16", 4, 2, 33, 17, 5, "tokens", [4, 6, 250], 21), ("bf16", "e4m3", 14, 2, 112, 112, 1, "tokens", [77, 1], 30),
    ("fp32", "e4m3", 4, 2, 96, 80, 8, "heads", [100], 6), ("bf16", "bf16", 4, 4, 128, 128, 16, "column", [20, 100], 3),
    ("bf16", "bf16", 2, 1, 160, 96, 16, "tokens", [4000], 200), ("bf16", "int8", 8, 4, 32, 32, 128, "tokens", [9000, 2049], 30),
    ("bf16", "bf16", 64, 8, 128, 128, 16, "tokens", [(389 * i) % 1500 for i in range(70)], 20),
]


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,lens,count", BLOCKS)
def test_block_attention(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, count):
    """Each cache head with a list of its own, in any order, with holes, the last block, ended lists."""
    t, b = T[dtype], len(lens)
    cache, table, slots, (kn, vn) = attention_case(dev, dtype, kind, heads, kv, dk, dv, page, order, lens)
    g = torch.Generator().manual_seed(7)
    blocks = torch.full((b, kv, count), -1, dtype=torch.int32)
    for i, n in enumerate(lens):
        many = -(-n // page)
        for h in range(kv):
            own = torch.randperm(max(many, 1), generator=g)[:min(many, count)].int()
            if h == 0 and many:
                own[-1] = many - 1                                      # the block that ends with the sequence (twice, perhaps)
            blocks[i, h, :len(own)] = own
    if b > 1 and lens[-1] > page:
        blocks[-1, 0, 0], blocks[-1, -1, min(1, count - 1)] = -1, 1 << 30
    q = rand((b, heads, dk), t, 11)
    out, lse = torch.full((b, heads, dv), -7.0, dtype=t, device=dev), torch.full((b, heads), -7.0, device=dev)
    Lq, Lo = f"({dk},{heads},{b}):(1,{dk},{heads * dk})", f"({dv},{heads},{b}):(1,{dv},{heads * dv})"
    lr.block_attention(q.to(dev), Lq, cache, blocks.to(dev), table.to(dev), int32(lens, dev), out, Lo, lse=lse)
    seen = [[blocks_seen(slots[i], blocks[i, h], lens[i], page) for h in range(kv)] for i in range(b)]
    want, wlse, tol = head_attention64(q, kn, vn, seen, kv, dk ** -0.5, t, kind)
    close(out, want, tol, "out")
    close(lse, wlse, tol.lse, "lse")


@pytest.mark.parametrize("dtype,kind,d", [("bf16", "bf16", 64), ("bf16", "e4m3", 64), ("bf16", "bf16", 33)])
def test_block_attention_lists(dev, dtype, kind, d):
    """Lists of nothing, of more entries than the sequence has blocks, of one block over and over, of blocks behind the
    sequence's end and past the table; lengths past the table; pages that are none."""
    t, heads, kv, page = T[dtype], 4, 2, 16
    lens = [100, 50, 33]
    cache, table, slots, (kn, vn) = attention_case(dev, dtype, kind, heads, kv, d, d, page, "tokens", lens)
    blocks = torch.tensor([[[-1] * 7, [3, 3, 3, 3, 3, 3, 3]],
                           [[0, 1, 2, 3, 3, 2, 1], [3, -2 ** 31, 2 ** 31 - 1, 0, 0, 0, 0]],
                           [[5, 3, 7, 0, 1, 2, 2], [2, 1, 0, 2, 1, 0, 2]]], dtype=torch.int32)
    q, L = rand((3, heads, d), t, 11), f"({d},{heads},3):(1,{d},{heads * d})"
    out, lse = torch.empty((3, heads, d), dtype=t, device=dev), torch.empty((3, heads), device=dev)
    lr.block_attention(q.to(dev), L, cache, blocks.to(dev), table.to(dev), int32(lens, dev), out, L, lse=lse)
    seen = [[blocks_seen(slots[i], blocks[i, h], lens[i], page) for h in range(kv)] for i in range(3)]
    want, wlse, tol = head_attention64(q, kn, vn, seen, kv, d ** -0.5, t, kind)
    close(out, want, tol)
    close(lse, wlse, tol.lse)
    assert (out[0, :2] == 0).all() and (lse[0, :2] == -math.inf).all()
    narrow = table[:, :3].clone()                                        # 48 tokens at most, whatever the lengths say
    narrow[0, 1] = -1
    lr.block_attention(q.to(dev), L, cache, blocks.to(dev), narrow.contiguous().to(dev), int32([100, 2 ** 31 - 1, -9], dev), out, L,
                       lse=lse)
    blocks[0] = torch.where(blocks[0] == 1, -1, blocks[0])
    seen = [[blocks_seen(slots[i], blocks[i, h], n, page) for h in range(kv)] for i, n in enumerate((48, 48, 0))]
    want, wlse, tol = head_attention64(q, kn, vn, seen, kv, d ** -0.5, t, kind)
    close(out, want, tol)
    close(lse, wlse, tol.lse)


def test_block_attention_of_all_is_paged_attention(dev):
    t, lens, heads, kv, d, page = torch.bfloat16, [700, 33, 0, 1600], 16, 4, 128, 16
    cache, table, slots, (kn, vn) = attention_case(dev, "bf16", "bf16", heads, kv, d, d, page, "heads", lens)
    q, L = rand((4, heads, d), t, 11).to(dev), f"({d},{heads},4):(1,{d},{heads * d})"
    blocks = torch.arange(100, dtype=torch.int32).expand(4, kv, 100).contiguous().to(dev)
    one, two = (torch.empty((4, heads, d), dtype=t, device=dev) for _ in range(2))
    lr.block_attention(q, L, cache, blocks, table.to(dev), int32(lens, dev), one, L)
    lr.paged_attention(q, L, cache, table.to(dev), int32(lens, dev), two, L)
    want, _, tol = attention64(q.cpu(), [kn[u] for u in slots], [vn[u] for u in slots], d ** -0.5, t, "bf16")
    close(one, want, tol)
    close(two, want, tol)


# ------------------------------------------------------------------------------------ together
def test_steps_on_streams_and_in_a_graph(dev):
    """Decoding steps as they would be used: positions of three axes, keys turned as they are stored, the blocks' keys,
    their choice and their attention, and attention over a shared prefix; on another stream, then captured and
    replayed with new inputs, against the same calls made eagerly."""
    b, h, kv, d, page, width, count = 3, 8, 2, 64, 16, 40, 6
    pages = b * width + 4
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).int().to(dev)
    table, prefix = perm[:b * width].view(b, width).contiguous(), perm[b * width:].contiguous()
    rt = lr.rope_axes_table(d, [12, 10, 10], order="cyclic", device=dev)
    L, Lk = lr.Layout(f"({d},{h},{b}):(1,{d},{h * d})"), lr.Layout(f"({d},{kv},{b}):(1,{d},{kv * d})")
    Lkeys = lr.Layout(f"({d},{kv},{pages}):(1,{d},{kv * d})")
    plen = int32([60], dev)

    def fresh():
        """A cache whose prefix and first tokens are written, and their blocks' keys."""
        k, v = (torch.zeros(pages * page * kv * d, dtype=torch.uint8, device=dev) for _ in range(2))
        ks, vs = (torch.zeros(pages * page * kv, device=dev) for _ in range(2))
        lay = f"({d},{kv},{page},{pages}):(1,{d},{kv * d},{page * kv * d})"
        cache = lr.PagedCache(k, lay, v, lay, ks, vs, f"({kv},{page},{pages}):(1,{kv},{page * kv})")
        n = 60 + 300 * b
        at = torch.arange(300, device=dev)
        slots = torch.cat([prefix.long()[at[:60] // page] * page + at[:60] % page]
                          + [table[i].long()[at // page] * page + at % page for i in range(b)])
        x = rand((n, kv, d), torch.bfloat16, 77).to(dev)
        Ln = f"({d},{kv},{n}):(1,{d},{kv * d})"
        lr.cache_write_axes(cache, x, Ln, x, Ln, slots, rt, ints(0, 500, (3, n), 6).to(dev))
        keys = torch.zeros((pages, kv, d), dtype=torch.bfloat16, device=dev)
        lr.block_keys(cache, slots, keys, Lkeys)
        return cache, keys

    def inputs(i):
        pos = torch.tensor([300 + i] * b, device=dev)
        q, k, v = (rand((b, n, d), torch.bfloat16, 100 * i + n + j).to(dev) for j, n in enumerate((h, kv, kv)))
        slots = table.long()[torch.arange(b, device=dev), pos // page] * page + pos % page
        return q, k, v, ints(0, 400, (3, b), i).to(dev), slots, (pos + 1).int()

    plans = (lr.prefix_attention_plan(L, fresh()[0], L, prefix.numel(), width, torch.bfloat16),
             lr.block_attention_plan(L, fresh()[0], L, count, torch.bfloat16), lr.block_select_plan(L, Lkeys, width))
    spaces = [torch.empty(max(p["workspace_bytes"], 1), dtype=torch.uint8, device=dev) for p in plans]

    def made():
        return (torch.empty((b, h, d), dtype=torch.bfloat16, device=dev), torch.empty((b, kv, count), dtype=torch.int32, device=dev),
                torch.empty((b, h, d), dtype=torch.bfloat16, device=dev), torch.empty((b, h, d), dtype=torch.bfloat16, device=dev))

    def step(held, x, out, ws, stream=None):
        (cache, keys), (q, k, v, pos, slots, lens), (qr, blocks, one, two) = held, x, out
        w = ws if ws else (None,) * 3
        lr.rope_axes(q, L, qr, L, pos, rt, stream=stream)
        lr.cache_write_axes(cache, k, Lk, v, Lk, slots, rt, pos, stream=stream)
        lr.block_keys(cache, slots, keys, Lkeys, stream=stream)
        lr.block_select(qr, L, keys, Lkeys, table, lens, page, blocks, workspace=w[2], stream=stream)
        lr.block_attention(qr, L, cache, blocks, table, lens, one, L, workspace=w[1], stream=stream)
        lr.prefix_attention(qr, L, cache, prefix, plen, table, lens, two, L, workspace=w[0], stream=stream)

    xs = [inputs(i) for i in range(5)]
    eager, want = fresh(), []
    for x in xs:
        want.append(made())
        step(eager, x, want[-1], spaces)
    torch.cuda.synchronize()
    # the choice and the attentions against 64 bits, from what the cache then holds
    cache, keys = eager
    q, blocks = want[-1][0].cpu(), want[-1][1].cpu()
    assert torch.equal(blocks, chosen64(q, keys.cpu(), table.cpu(), [305] * b, page, count, 1, 1))
    info = ("tokens", pages, page, kv, 0)
    kn, vn = (c.to(F64) * s.to(F64)[..., None] for c, s in (content(cache, info, d, w) for w in ("k", "v")))
    at = torch.arange(305)
    slots = [table[i].cpu().long()[at // page] * page + at % page for i in range(b)]
    seen = [[blocks_seen(slots[i], blocks[i, g], 305, page) for g in range(kv)] for i in range(b)]
    exact, _, tol = head_attention64(q, kn, vn, seen, kv, d ** -0.5, torch.bfloat16, "e4m3")
    close(want[-1][2], exact, tol, "blocks")
    shared = prefix.cpu().long()[at[:60] // page] * page + at[:60] % page
    seen = [torch.cat([shared, u]) for u in slots]
    exact, _, tol = attention64(q, [kn[u] for u in seen], [vn[u] for u in seen], d ** -0.5, torch.bfloat16, "e4m3")
    close(want[-1][3], exact, tol, "prefix")
    # another stream, workspaces allocated by the calls
    side, held = torch.cuda.Stream(), fresh()
    for i, x in enumerate(xs):
        out = made()
        torch.cuda.synchronize()
        step(held, x, out, None, stream=side)
        side.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(out, want[i])), i
    # a graph, its inputs copied in before each replay
    held, x, out = fresh(), [z.clone() for z in xs[0]], made()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held, x, out, spaces)
    for i in range(5):
        for dst, src in zip(x, xs[i]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(out, want[i])), i
        torch.randn(1 << 20, device=dev).sum().item()                    # eager work between the replays


def test_steps_of_no_sequence(dev):
    """A step whose batch has become empty runs through all entry points and writes nothing."""
    d, h, kv, page, pages, width = 64, 4, 2, 16, 6, 3
    L, Lk, Lkeys = f"({d},{h},1):(1,{d},{h * d})", f"({d},{kv},1):(1,{d},{kv * d})", f"({d},{kv},{pages}):(1,{d},{kv * d})"
    rt = lr.rope_axes_table(d, [16, 8, 8], device=dev)
    cache, _ = make_cache(dev, "bf16", "tokens", pages, page, kv, d, d)
    one = torch.ones((1, h, d), dtype=torch.bfloat16, device=dev)
    k, keys = torch.ones((1, kv, d), dtype=torch.bfloat16, device=dev), torch.full((pages, kv, d), 3.0, dtype=torch.bfloat16, device=dev)
    table, lens = torch.zeros((0, width), dtype=torch.int32, device=dev), int32([], dev)
    slots, pos = torch.empty(0, dtype=torch.int64, device=dev), torch.empty((3, 0), dtype=torch.int64, device=dev)
    outs = [torch.full_like(one, 7.0) for _ in range(3)]
    blocks = torch.empty((0, kv, 4), dtype=torch.int32, device=dev)
    before = cache.k.clone()
    lr.rope_axes(one, L, outs[0], L, pos, rt)
    lr.cache_write_axes(cache, k, Lk, k, Lk, slots, rt, pos)
    lr.block_keys(cache, slots, keys, Lkeys)
    lr.block_select(one, L, keys, Lkeys, table, lens, page, blocks)
    lr.block_attention(one, L, cache, blocks, table, lens, outs[1], L)
    lr.prefix_attention(one, L, cache, int32([0, 1], dev), int32([20], dev), table, lens, outs[2], L)
    torch.cuda.synchronize()
    assert all((x == 7.0).all() for x in outs) and (keys == 3.0).all() and torch.equal(cache.k, before)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_past_32_bits(dev, kind):
    """Pages 2^30 elements apart, the last one past 2^32: the same results as with pages next to each other."""
    d, h, page, pages, b, step = 64, 4, 2048, 5, 32, 1 << 30
    t = T[kind] if kind == "bf16" else torch.uint8
    L, n = f"({d},{h},{b}):(1,{d},{h * d})", pages * page
    Ls, Ln = f"(1,{page},{pages}):(1,1,{page})", f"({d},1,{n}):(1,{d},{d})"
    rt = lr.rope_axes_table(d, [16, 8, 8], device=dev)
    k, v = (rand((n, 1, d), torch.bfloat16, s).to(dev) for s in (1, 2))
    q, pos = rand((b, h, d), torch.bfloat16, 3).to(dev), ints(0, 90, (3, n), 4).to(dev)
    slots = torch.arange(n, device=dev)
    table = torch.randperm(pages * b, generator=torch.Generator().manual_seed(5)).int().view(b, pages).to(dev) % pages
    lens = int32([n - 37 * i for i in range(b)], dev)
    prefix = int32([4, 1, 0, 3, 2], dev)

    def run(stride):
        size = (pages - 1) * stride + page * d
        bufs = [torch.empty(size, dtype=t, device=dev) for _ in range(2)]
        Lc = f"({d},1,{page},{pages}):(1,{d},{d},{stride})"
        scales = [torch.empty(n, device=dev) for _ in range(2)] if kind != "bf16" else [None, None]
        cache = lr.PagedCache(bufs[0], Lc, bufs[1], Lc, *scales, Ls if kind != "bf16" else None)
        lr.cache_write_axes(cache, k, Ln, v, Ln, slots, rt, pos)
        keys = torch.empty((pages - 1) * stride + d, dtype=torch.bfloat16, device=dev)
        Lkeys = f"({d},1,{pages}):(1,{d},{stride})"
        lr.block_keys(cache, slots, keys, Lkeys)
        blocks = torch.empty((b, 1, 3), dtype=torch.int32, device=dev)
        lr.block_select(q, L, keys, Lkeys, table, lens, page, blocks)
        outs = [torch.empty_like(q) for _ in range(3)]
        lr.block_attention(q, L, cache, blocks, table, lens, outs[0], L)
        lr.prefix_attention(q, L, cache, prefix, int32([n - 5], dev), table, lens, outs[1], L)  # 128 rows share tiles
        L4 = f"({d},{h},4):(1,{d},{h * d})"
        lr.prefix_attention(q, L4, cache, prefix, int32([n - 5], dev), table, lens[:4], outs[2], L4)
        outs[2][4:] = 0
        last = keys.as_strided((pages, d), (stride, 1)).clone()
        turned = torch.empty_like(last)
        lr.rope_axes(keys, Lkeys, turned, f"({d},1,{pages}):(1,{d},{d})", pos[:, :pages].contiguous(), rt)
        return [blocks, *outs, last, turned]

    near = run(page * d)
    for i, (x, y) in enumerate(zip(near, run(step))):
        assert torch.equal(x, y), i
    assert near[1].isfinite().all() and near[1].abs().max() > 0 and near[2].isfinite().all()


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,b,prefix", [
    ("bf16", "bf16", 8, 2, 128, 128, 16, 330, 700), ("fp16", "e4m3", 6, 2, 96, 96, 16, 431, 90), ("fp32", "fp32", 7, 7, 33, 33, 5, 367, 50),
    ("bf16", "int8", 4, 1, 64, 256, 8, 643, 0), ("fp16", "fp16", 64, 8, 64, 4, 16, 41, 3000), ("fp32", "fp32", 5, 1, 8, 250, 4, 515, 61)])
def test_prefix_attention_many_heads(dev, dtype, kind, heads, kv, dk, dv, page, b, prefix):
    """So many heads that a wave joins each one's parts: widths that leave lanes without a column, heads that do not
    fill the last workgroup, rows without a sequence, rows behind the batch."""
    t = T[dtype]
    assert b * heads >= 2560
    lens = [(37 * i) % 53 if i % 101 else 900 for i in range(b)]
    cache, first, table, shared, slots, (kn, vn) = prefix_case(dev, dtype, kind, heads, kv, dk, dv, page, "tokens", prefix, lens)
    q = rand((b, heads, dk), t, 11)
    none = [5, b - 2]
    given = [-1 if i in none else n for i, n in enumerate(lens)]
    out = torch.full((b + 1, heads, dv), -7.0, dtype=t, device=dev)
    lse = torch.full((b + 1, heads), -7.0, device=dev)
    lr.prefix_attention(q.to(dev), f"({dk},{heads},{b}):(1,{dk},{heads * dk})", cache, first.to(dev), int32([prefix], dev),
                        table.to(dev), int32(given, dev), out, f"({dv},{heads},{b}):(1,{dv},{heads * dv})", lse=lse)
    assert (out[b] == -7).all() and (lse[b] == -7).all()
    assert (out[none] == 0).all() and (lse[none] == -math.inf).all()
    some = [i for i in sorted({*range(0, b, max(1, b // 12)), 101, b - 1}) if i < b and i not in none]
    seen = [torch.cat([shared, slots[i]]) for i in some]
    want, wlse, tol = attention64(q[some], [kn[u] for u in seen], [vn[u] for u in seen], dk ** -0.5, t, kind)
    close(out.cpu()[some], want, tol, "out")
    close(lse.cpu()[some], wlse, tol.lse, "lse")


@pytest.mark.parametrize("dtype,kind,dim,page,width", [("bf16", "bf16", 128, 16, 512), ("fp16", "fp16", 64, 8, 600),
                                                       ("bf16", "e4m3", 96, 32, 300), ("fp16", "int8", 128, 16, 513)])
def test_prefix_attention_beside_long_sequences(dev, dtype, kind, dim, page, width):
    """A prefix whose rows share tiles, in one launch with own tokens that four cache heads of a workgroup read."""
    t, heads, kv, b, prefix = T[dtype], 32, 8, 32, 700
    lens = [(97 * i) % 211 for i in range(b)]
    lens[3], lens[20] = 1024, 777
    assert b * heads // kv * width * page >= (1 << 20 if kind in TOP else 600000)
    cache, first, table, shared, slots, (kn, vn) = prefix_case(dev, dtype, kind, heads, kv, dim, dim, page, "tokens", prefix, lens)
    wide = torch.full((width,), -1, dtype=torch.int32)
    wide[:-(-prefix // page)] = first[:-(-prefix // page)]
    q, L = rand((b, heads, dim), t, 11), f"({dim},{heads},{b}):(1,{dim},{heads * dim})"
    out, lse = torch.full((b, heads, dim), -7.0, dtype=t, device=dev), torch.full((b, heads), -7.0, device=dev)
    given = [-1 if i == 7 else n for i, n in enumerate(lens)]
    lr.prefix_attention(q.to(dev), L, cache, wide.to(dev), int32([prefix], dev), table.to(dev), int32(given, dev), out, L, lse=lse)
    assert (out[7] == 0).all() and (lse[7] == -math.inf).all()
    some = [0, 1, 3, 8, 20, 31]
    seen = [torch.cat([shared, slots[i]]) for i in some]
    want, wlse, tol = attention64(q[some], [kn[u] for u in seen], [vn[u] for u in seen], dim ** -0.5, t, kind)
    close(out.cpu()[some], want, tol, "out")
    close(lse.cpu()[some], wlse, tol.lse, "lse")
