"""The operators for long and many-sided contexts on the GPU against plain 64-bit forms computed here on the CPU.

Tolerances count roundings: storing a value in type T is off by at most half a step, HALF[T] relative
(or half the smallest subnormal), and every 32-bit operation by 2^-24 of its result.
"""

import math

import pytest

torch = pytest.importorskip("torch")
import layout_remapping_copy_amd as lr  # noqa: E402

pytestmark = pytest.mark.gpu

F64 = torch.float64
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
T = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
     "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lr.lib()
    return torch.device("cuda:0")


def close(got, want, tol, what=""):
    got, want = got.to(F64).cpu(), want.to(F64)
    assert got.shape == want.shape
    same = (got == want) | (got.isnan() & want.isnan())
    off = (got - want).abs()
    bad = ~same & ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(off[bad][0]), float((tol.expand_as(off) if torch.is_tensor(tol) else
                                                                           torch.tensor(tol).expand_as(off))[bad][0]))


def rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float32).to(dtype)


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


def rope_tolerance(want, size, dtype):
    # cos and sin 2^-23 off, one rounding each for the magnitude, the products and the sum
    return HALF[dtype] * want.abs() + 8 * U * size + TINY[dtype]


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
def cache_strides(order, h, p, d, pad=0):
    """(pages, slots, heads, dim) strides of a cache tensor and (pages, slots, heads) of its scales."""
    r = d + pad
    if order == "tokens":
        return (p * h * r, h * r, r, 1), (p * h, h, 1)
    if order == "heads":
        return (h * p * r, r, p * r, 1), (h * p, 1, p)
    return (h * p * d, 1, p, h * p), (p * h, h, 1)      # "column": the head dimension outermost in a page


def make_cache(dev, kind, order, pages, p, h, dk, dv, pad=0):
    t = T[kind]
    tensors, layouts = [], []
    for d in (dk, dv):
        s, ss = cache_strides(order, h, p, d, pad)
        n = 1 + (pages - 1) * s[0] + (p - 1) * s[1] + (h - 1) * s[2] + (d - 1) * s[3]
        tensors.append(torch.zeros(n, dtype=t if kind != "e4m3" else torch.uint8, device=dev))
        layouts.append(f"({d},{h},{p},{pages}):({s[3]},{s[2]},{s[1]},{s[0]})")
    ks = vs = Ls = None
    if kind in TOP:
        ks, vs = (torch.full((pages * p * h,), -1.0, device=dev) for _ in range(2))
        Ls = f"({h},{p},{pages}):({ss[2]},{ss[1]},{ss[0]})"
    return lr.PagedCache(tensors[0], layouts[0], tensors[1], layouts[1], ks, vs, Ls), (order, pages, p, h, pad)


def content(cache, info, d, which):
    """(codes as their values, scales or None) of a cache side as (pages * slots, heads, ...), on the CPU."""
    order, pages, p, h, pad = info
    s, ss = cache_strides(order, h, p, d, pad)
    x = getattr(cache, which).cpu().as_strided((pages, p, h, d), s).reshape(pages * p, h, d)
    if x.dtype == torch.uint8:
        x = x.contiguous().view(torch.float8_e4m3fn).float()
    sc = getattr(cache, which + "_scale")
    return x, None if sc is None else sc.cpu().as_strided((pages, p, h), ss).reshape(pages * p, h)


def stored(cache, info, d, which):
    """What the cache stands for, in 64 bits."""
    x, s = content(cache, info, d, which)
    return x.to(F64) if s is None else x.to(F64) * s.to(F64)[..., None]


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
