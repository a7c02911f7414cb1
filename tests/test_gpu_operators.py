"""The attention operators on the GPU against plain 64-bit forms computed here on the CPU.

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


def buffer(x, shape_strides, dev, fill=0.0, extra=0):
    """x (logical dims) laid into a flat GPU buffer by strides; returns (buffer, view)."""
    n = 1 + sum((s - 1) * d for s, d in zip(x.shape, shape_strides)) + extra
    flat = torch.full((n,), fill, dtype=x.dtype)
    flat.as_strided(x.shape, shape_strides).copy_(x)
    return flat.to(dev)


# ------------------------------------------------------------------------------------ rotary positions
def rotate64(x, positions, table, pairs, sign=1):
    """x (tokens, heads, dim) in 64 bits; the angle from the table's fractions of a turn, exactly."""
    rot, turns, m = table.rot_dim, table.turns.cpu(), table.magnitude
    frac = (positions.reshape(-1, 1) * turns).to(F64) / 2.0 ** 64     # int64 product wraps: whole turns drop out
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


ROPE = [  # dtype, tokens, heads, dim, rot, pairs, token stride of y (None: as x), scaling
    ("bf16", 7, 3, 128, 128, "half", None), ("bf16", 7, 3, 128, 128, "interleaved", None),
    ("fp16", 1, 1, 64, 64, "half", None), ("fp32", 65, 5, 80, 32, "interleaved", None),
    ("bf16", 33, 2, 72, 36, "half", None), ("fp16", 33, 2, 72, 18, "half", None), ("fp32", 9, 4, 20, 6, "interleaved", None),
    ("bf16", 5, 2, 33, 16, "half", None), ("fp16", 5, 2, 33, 22, "interleaved", None), ("fp32", 1, 1, 2, 2, "half", None),
    ("bf16", 130, 40, 96, 64, "half", "heads"), ("fp16", 130, 8, 256, 256, "interleaved", "heads"),
    ("bf16", 257, 4, 1024, 1024, "half", "heads"), ("fp32", 1030, 1, 128, 128, "half", "heads"),
    ("bf16", 13, 3, 24, 8, "half", "column"), ("fp32", 13, 3, 24, 8, "interleaved", "column"),
]


@pytest.mark.parametrize("dtype,n,h,d,rot,pairs,order", ROPE)
def test_rope(dev, dtype, n, h, d, rot, pairs, order):
    t = T[dtype]
    x = rand((n, h, d), t, n + d)
    positions = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(1))
    table = lr.rope_table(rot, base=500000.0, scaling="bands", factor=8.0, original_len=8192, low=1.0, high=4.0, device=dev)
    sx = (h * d, d, 1)
    sy = {None: sx, "heads": (d, n * d, 1), "column": (1, n * d, n)}[order]
    for backward in (False, True):
        y = torch.full((n * h * d,), -7.0, dtype=t, device=dev)
        lr.rope(x.to(dev), f"({d},{h},{n}):(1,{d},{h * d})", y, f"({d},{h},{n}):({sy[2]},{sy[1]},{sy[0]})",
                positions.to(dev), table, pairs=pairs, backward=backward)
        want, size = rotate64(x, positions, table, pairs, -1 if backward else 1)
        close(y.cpu().as_strided((n, h, d), sy), want, rope_tolerance(want, size, t), backward)


def test_rope_far_positions(dev):
    """Angles stay exact at any int64 position, negative ones included."""
    pos = torch.tensor([0, 1, -1, 131071, 10 ** 6, 10 ** 9, -10 ** 9, 2 ** 40 + 1, 2 ** 62, -2 ** 63, 2 ** 63 - 1])
    x = rand((len(pos), 2, 64), torch.float32, 3)
    table = lr.rope_table(64, device=dev)
    y = torch.empty(x.shape, device=dev)
    L = f"(64,2,{len(pos)}):(1,64,128)"
    lr.rope(x.to(dev), L, y, L, pos.to(dev), table)
    want, size = rotate64(x, pos, table, "half")
    close(y, want, rope_tolerance(want, size, torch.float32))
    # and the table's frequencies against the formula, at a position where 32-bit angles have long lost theirs
    a = 131071 * 10000.0 ** (-torch.arange(32, dtype=F64) / 32)
    p, q = x[3, 0, :32].to(F64), x[3, 0, 32:].to(F64)
    close(y[3, 0, :32], p * a.cos() - q * a.sin(), 1e-6 * (p.abs() + q.abs()))


@pytest.mark.parametrize("aligned", [True, False])
def test_rope_shared_positions_and_padding(dev, aligned):
    """Positions shared over a batch (stride 0), tokens of several leaves, padded rows, a part of the tokens,
    an offset buffer; what the layout does not reach stays as it was."""
    b, n, h, d = 3, 11, 4, 32
    row = d + (8 if aligned else 3)
    x = rand((b, n, h, d), torch.bfloat16, 5)
    xb = buffer(x, (n * h * row, h * row, row, 1), dev, fill=float("nan"))
    table = lr.rope_table(16, device=dev)
    pos = torch.randint(0, 5000, (n,), generator=torch.Generator().manual_seed(2))
    y = torch.full((b * h * n * row + 1,), -7.0, dtype=torch.bfloat16, device=dev)
    Lx = f"({d},{h},({n},{b})):(1,{row},({h * row},{n * h * row}))"
    Ly = f"({d},{h},({n},{b})):(1,{n * row},({row},{h * n * row}))"
    used = 2 * n + 4
    off = 0 if aligned else 1
    lr.rope(xb, Lx, y[off:], Ly, pos.to(dev), table, Lp=f"({n},{b}):(1,0)", n=used)
    want, size = rotate64(x.reshape(b * n, h, d), pos.repeat(b), table, "half")
    got = y.cpu()[off:].as_strided((b, h, n, d), (h * n * row, n * row, row, 1)).permute(0, 2, 1, 3).reshape(b * n, h, d)
    close(got[:used], want[:used], rope_tolerance(want, size, torch.bfloat16)[:used])
    assert (got[used:] == -7).all()
    assert int((y == -7).sum()) == y.numel() - used * h * d


def test_rope_in_place(dev):
    for dtype, d in (("bf16", 128), ("fp32", 30)):
        x = rand((50, 3, d), T[dtype], 7).to(dev)
        L = f"({d},3,50):(1,{d},{3 * d})"
        pos = torch.arange(50, device=dev)
        table = lr.rope_table(d, device=dev)
        y = lr.rope(x, L, torch.empty_like(x), L, pos, table)
        lr.rope(x, L, x, L, pos, table)
        assert torch.equal(x, y)


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
def test_rope_gradient_by_differences(dev, pairs):
    """The loss sum(w y^2)/2 is quadratic in x, so its central difference along a direction is the gradient's
    product with it for any step; with the gradient R^T (w y) from the backward call."""
    n, h, d, rot = 37, 3, 48, 32
    x, w, e = (rand((n, h, d), torch.float32, s).to(dev) for s in (1, 2, 3))
    L = f"({d},{h},{n}):(1,{d},{h * d})"
    pos = torch.arange(n, device=dev) * 1000
    table = lr.rope_table(rot, scaling="parts", factor=4.0, original_len=2048, device=dev)

    def forward(z):
        return lr.rope(z, L, torch.empty_like(z), L, pos, table, pairs=pairs)
    y = forward(x)
    grad = lr.rope(w * y, L, torch.empty_like(x), L, pos, table, pairs=pairs, backward=True)
    up, down = forward(x + e).double(), forward(x - e).double()
    got = ((w.double() * (up ** 2 - down ** 2)).sum() / 4).item()
    want = (grad.double() * e.double()).sum().item()
    terms = (w.double().abs() * (up ** 2 + down ** 2)).sum().item() / 4 + (grad.double() * e.double()).abs().sum().item()
    assert abs(got - want) <= 16 * U * terms


def test_rope_nan_and_infinity(dev):
    x = rand((4, 1, 16), torch.float32, 1)
    x[0, 0, 0], x[1, 0, 3], x[2, 0, 15] = float("nan"), float("inf"), float("-inf")
    L = "(16,1,4):(1,16,16)"
    table = lr.rope_table(8, device=dev)
    y = lr.rope(x.to(dev), L, torch.empty((4, 1, 16), device=dev), L, torch.ones(4, dtype=torch.int64, device=dev), table).cpu()
    assert y[0, 0, 0].isnan() and y[0, 0, 4].isnan() and y[0].isnan().sum() == 2
    assert y[1, 0, 3].isinf() and y[1, 0, 7].isinf() and y[2, 0, 15] == float("-inf")


# ------------------------------------------------------------------------------------ the cache
def cache_strides(order, h, p, d, pad=0):
    """(pages, slots, heads, dim) strides of a cache tensor and (pages, slots, heads) of its scales."""
    r = d + pad
    if order == "tokens":
        return (p * h * r, h * r, r, 1), (p * h, h, 1)
    if order == "heads":
        return (h * p * r, r, p * r, 1), (h * p, 1, p)
    return (h * p * d, 1, p, h * p), (p * h, h, 1)      # "column": the head dimension outermost in a page


def make_cache(dev, kind, order, pages, p, h, dk, dv, pad=0, fill=None):
    t = T[kind]
    tensors, layouts = [], []
    for d in (dk, dv):
        s, ss = cache_strides(order, h, p, d, pad)
        n = 1 + (pages - 1) * s[0] + (p - 1) * s[1] + (h - 1) * s[2] + (d - 1) * s[3]
        raw = torch.zeros(n, dtype=t if kind != "e4m3" else torch.uint8)
        if fill is not None:
            raw.fill_(fill)
        tensors.append(raw.to(dev))
        layouts.append(f"({d},{h},{p},{pages}):({s[3]},{s[2]},{s[1]},{s[0]})")
    ks = vs = Ls = None
    if kind in ("e4m3", "int8"):
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


def nearest_e4m3(x):
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (x / step).round() * step


TOP = {"e4m3": 448.0, "int8": 127.0}


def quantised64(x, kind):
    """Codes (as values) and scales by the definition: 32-bit scale, the exact quotient rounded to nearest even."""
    fin = torch.where(x.isfinite(), x, torch.zeros_like(x))
    scale = (fin.abs().amax(-1).float() / TOP[kind]).clamp(min=2.0 ** -126)
    q = (x.to(F64) / scale.to(F64)[..., None]).clamp(-TOP[kind], TOP[kind])
    return (nearest_e4m3(q) if kind == "e4m3" else q.nan_to_num(0).round()), scale


CACHE = [  # type, kind, tokens, heads, dk, dv, page, order, pad
    ("bf16", "e4m3", 1, 1, 128, 128, 16, "tokens", 0), ("bf16", "e4m3", 77, 8, 128, 128, 16, "heads", 0),
    ("fp16", "int8", 77, 4, 96, 96, 16, "tokens", 0), ("fp32", "e4m3", 33, 3, 80, 64, 5, "heads", 0),
    ("fp32", "int8", 33, 3, 20, 36, 1, "tokens", 4), ("bf16", "int8", 40, 2, 33, 65, 7, "tokens", 3),
    ("fp16", "e4m3", 40, 2, 512, 256, 64, "heads", 16), ("bf16", "bf16", 50, 5, 128, 192, 32, "heads", 8),
    ("fp16", "fp16", 50, 5, 72, 72, 8, "tokens", 0), ("fp32", "fp32", 50, 2, 256, 256, 16, "tokens", 0),
    ("bf16", "e4m3", 300, 2, 64, 64, 16, "column", 0), ("fp16", "int8", 2000, 8, 128, 128, 16, "tokens", 0),
    ("bf16", "e4m3", 2000, 16, 256, 256, 128, "heads", 0), ("fp32", "fp32", 21, 1, 7, 3, 3, "column", 0),
    ("bf16", "int8", 64, 2, 400, 300, 16, "heads", 0), ("bf16", "bf16", 64, 2, 40, 44, 16, "tokens", 0),
]


def new_slots(n, pages, p, seed, missing=0):
    g = torch.Generator().manual_seed(seed)
    slots = torch.randperm(pages * p, generator=g)[:n].clone()
    if missing:
        bad = torch.tensor([-1, pages * p, -2 ** 62, 2 ** 62, 2 ** 32])
        slots[torch.randperm(n, generator=g)[:missing]] = bad[torch.arange(missing) % 5]
    return slots


@pytest.mark.parametrize("dtype,kind,n,h,dk,dv,page,order,pad", CACHE)
def test_cache_write_and_read(dev, dtype, kind, n, h, dk, dv, page, order, pad):
    t, pages = T[dtype], -(-n // page) + 2
    k, v = rand((n, h, dk), t, 1) * 3, rand((n, h, dv), t, 2)
    if n > 8:
        k[1], v[2] = 0, 2.0 ** -133                       # rows of zeros and of tiny values
        k[3, 0, 0], k[4, 0, 1], v[5, 0, 2] = float("inf"), float("-inf"), float("nan")
    slots = new_slots(n, pages, page, 3, missing=5 if n > 8 else 0)
    cache, info = make_cache(dev, kind, order, pages, page, h, dk, dv, pad)
    Lk, Lv = f"({dk},{h},{n}):(1,{dk},{h * dk})", f"({dv},{h},{n}):(1,{dv},{h * dv})"
    lr.cache_write(cache, k.to(dev), Lk, v.to(dev), Lv, slots.to(dev))
    keep = (slots >= 0) & (slots < pages * page)
    ko, vo = (torch.full((n, h, d), -7.0, dtype=t, device=dev) for d in (dk, dv))
    lr.cache_read(cache, slots.to(dev), ko, Lk, vo, Lv)
    for x, d, which, back in ((k, dk, "k", ko), (v, dv, "v", vo)):
        got, scales = content(cache, info, d, which)
        if kind in TOP:
            codes, scale = quantised64(x, kind)
            want = torch.zeros(got.shape, dtype=F64)
            want[slots[keep]] = codes[keep]
            close(got, want, 0.0, which)                   # the codes are exact, ties included
            ws = torch.full(scales.shape, -1.0, dtype=F64)
            ws[slots[keep]] = scale[keep].to(F64)
            close(scales, ws, 0.0, which + " scales")
            full = codes * scale.to(F64)[..., None]
            tol = (HALF[t] + U) * full.abs() + TINY[t]
        else:
            want = torch.zeros(got.shape, dtype=F64)
            want[slots[keep]] = x[keep].to(F64)
            close(got, want, 0.0, which)
            full, tol = x.to(F64), 0.0
        full = torch.where(keep[:, None, None], full, torch.zeros_like(full))
        close(back, full, tol, which + " read")


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,kind,n,h,d,rot,page", [("bf16", "e4m3", 70, 8, 128, 128, 16), ("fp16", "int8", 33, 2, 96, 64, 16),
                                                      ("fp32", "fp32", 9, 3, 80, 16, 5), ("bf16", "bf16", 40, 4, 64, 64, 8),
                                                      ("bf16", "e4m3", 20, 2, 72, 36, 16), ("bf16", "e4m3", 20, 2, 33, 16, 16),
                                                      ("fp16", "e4m3", 1000, 8, 256, 128, 64), ("bf16", "int8", 3, 1, 512, 512, 4)])
def test_cache_write_rotated(dev, pairs, dtype, kind, n, h, d, rot, page):
    t, pages = T[dtype], -(-n // page) + 1
    k, v = rand((n, h, d), t, 1), rand((n, h, d), t, 2)
    pos = torch.randint(0, 100000, (n,), generator=torch.Generator().manual_seed(9))
    table = lr.rope_table(rot, scaling="parts", factor=4.0, original_len=4096, device=dev)
    slots = new_slots(n, pages, page, 4)
    cache, info = make_cache(dev, kind, "tokens", pages, page, h, d, d)
    L = f"({d},{h},{n}):(1,{d},{h * d})"
    lr.cache_write(cache, k.to(dev), L, v.to(dev), L, slots.to(dev), table=table, positions=pos.to(dev), pairs=pairs)
    want, size = rotate64(k, pos, table, pairs)
    got, scales = content(cache, info, d, "k")
    got = got[slots].to(F64)
    if kind in TOP:
        s = scales[slots].to(F64)[..., None]
        close(scales[slots], want.abs().amax(-1) / TOP[kind], 10 * U * (size.amax(-1) + want.abs().amax(-1)) / TOP[kind])
        half = (got.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) if kind == "e4m3" else torch.full_like(got, 0.5)
        close(got * s, want, half * s * (1 + 2.0 ** -20) + 12 * U * (size + want.abs().amax(-1, keepdim=True)))
        codes, _ = quantised64(v, kind)
        close(content(cache, info, d, "v")[0][slots], codes, 0.0)
    else:
        close(got, want, rope_tolerance(want, size, t))
        close(content(cache, info, d, "v")[0][slots], v.to(F64), 0.0)


def test_cache_beyond_32_bits(dev):
    """Offsets of 2^32 elements and more on both sides."""
    pages, p, h, d = 33000, 64, 8, 256           # 4.3e9 elements a tensor
    k, v = (torch.empty(pages * p * h * d, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.empty(pages * p * h, device=dev) for _ in range(2))
    L = f"({d},{h},{p},{pages}):(1,{d},{h * d},{p * h * d})"
    cache = lr.PagedCache(k, L, v, L, ks, vs, f"({h},{p},{pages}):(1,{h},{p * h})")
    slots = torch.tensor([0, 5, pages * p - 1, pages * p - 70, 32768 * 64, 32768 * 64 - 1])
    n = len(slots)
    x, y = rand((n, h, d), torch.bfloat16, 1), rand((n, h, d), torch.bfloat16, 2)
    Lx = f"({d},{h},{n}):(1,{d},{h * d})"
    lr.cache_write(cache, x.to(dev), Lx, y.to(dev), Lx, slots.to(dev))
    a, b = (torch.empty((n, h, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
    lr.cache_read(cache, slots.to(dev), a, Lx, b, Lx)
    for z, w in ((x, a), (y, b)):
        codes, scale = quantised64(z, "e4m3")
        full = codes * scale.to(F64)[..., None]
        close(w, full, (HALF[torch.bfloat16] + U) * full.abs())
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device=dev)
    # the last page of a long cache holds whatever memory held; give it numbers
    fresh = rand((p, h, d), torch.float32, 8)
    c8, s8 = quantised64(fresh, "e4m3")
    k.view(pages, p, h, d)[pages - 1] = c8.float().to(torch.float8_e4m3fn).view(torch.uint8).to(dev)
    v.view(pages, p, h, d)[pages - 1] = c8.float().to(torch.float8_e4m3fn).view(torch.uint8).to(dev)
    ks.view(pages, p, h)[pages - 1], vs.view(pages, p, h)[pages - 1] = s8.to(dev), s8.to(dev)
    q = rand((1, h, d), torch.bfloat16, 3)
    out = torch.empty((1, h, d), dtype=torch.bfloat16, device=dev)
    Lq = f"({d},{h},1):(1,{d},{h * d})"
    lr.paged_attention(q.to(dev), Lq, cache, table, torch.tensor([p], dtype=torch.int32, device=dev), out, Lq)
    val = c8 * s8.to(F64)[..., None]
    want, _, tol = attention64(q, [val], [val], d ** -0.5, T["bf16"], "e4m3")
    close(out, want, tol)


# ------------------------------------------------------------------------------------ attention
def attention64(q, ks, vs, scale, dtype, kind):
    """q (b, heads, dk), and per sequence the seen keys and values (t, kv heads, d) as 64-bit numbers.
    Returns out, lse and out's tolerance (lse's as an attribute of the tensor returned last)."""
    b, h, _ = q.shape
    dv = vs[0].shape[-1]
    out, tol = torch.zeros((b, h, dv), dtype=F64), torch.zeros((b, h, dv), dtype=F64)
    lse, ltol = torch.full((b, h), -math.inf, dtype=F64), torch.zeros((b, h), dtype=F64)
    # the weights meet the values in the matrix type: the model's, or bf16 for 8-bit caches
    weight = HALF[dtype] if dtype == torch.float32 else HALF[torch.bfloat16] if kind in TOP else HALF[dtype]
    for i in range(b):
        n, g = ks[i].shape[0], h // ks[i].shape[1]
        if n == 0:
            continue
        k, v = (x[i].to(F64).repeat_interleave(g, 1).transpose(0, 1) for x in (ks, vs))   # (heads, t, d)
        x = q[i].to(F64)
        s = torch.einsum("hd,htd->ht", x, k) * scale
        p = torch.softmax(s, -1)
        out[i] = torch.einsum("ht,htd->hd", p, v)
        lse[i] = torch.logsumexp(s, -1)
        # a score: as many 32-bit roundings as products, of the terms' sizes; a weight: twice that and the exponential's
        ds = (torch.einsum("hd,htd->ht", x.abs(), k.abs()) * abs(scale)).amax(-1) * (k.shape[-1] + 8) * U
        sums = (n + 16) * U
        size = torch.einsum("ht,htd->hd", p, v.abs())
        # fp16 weights below 2^-14 lose bits: at most half their smallest step, relative to a largest weight of 1
        small = n * 2.0 ** -25 * v.abs().amax(1) if dtype == torch.float16 and kind not in TOP else 0.0
        tol[i] = HALF[dtype] * out[i].abs() + (weight + sums + 2 * ds[:, None] + 2.0 ** -20) * size + small + TINY[dtype]
        ltol[i] = ds + sums + 2.0 ** -20 + 2.0 ** -22 * lse[i].abs()
    tol.lse = ltol
    return out, lse, tol


ATTEND = [  # type, kind, heads, kv, dk, dv, page, order, lens, window
    ("bf16", "bf16", 8, 2, 128, 128, 16, "tokens", [1, 15, 16, 17, 0, 129, 700], 0),
    ("fp16", "fp16", 8, 8, 64, 64, 16, "heads", [1, 2, 31, 32, 33, 500], 0),
    ("fp32", "fp32", 6, 3, 128, 128, 16, "tokens", [1, 0, 65, 300], 0),
    ("bf16", "e4m3", 32, 8, 128, 128, 64, "heads", [1, 63, 64, 65, 1000], 0),
    ("fp16", "int8", 20, 1, 80, 80, 32, "tokens", [1, 40, 900], 100),
    ("fp32", "int8", 5, 1, 64, 64, 16, "tokens", [3, 100], 0),
    ("fp32", "e4m3", 4, 2, 96, 80, 8, "heads", [3, 100], 33),
    ("bf16", "bf16", 16, 1, 192, 128, 16, "tokens", [0, 257, 64], 0),
    ("bf16", "bf16", 48, 1, 256, 256, 16, "heads", [200, 31], 0),
    ("fp16", "fp16", 7, 1, 72, 72, 8, "tokens", [9, 333], 0),
    ("bf16", "bf16", 4, 2, 33, 17, 5, "tokens", [1, 4, 5, 6, 250], 0),
    ("bf16", "e4m3", 14, 2, 112, 112, 1, "tokens", [77, 1], 0),
    ("fp16", "int8", 8, 2, 160, 160, 7, "heads", [50, 300], 1),
    ("bf16", "bf16", 4, 4, 128, 128, 16, "column", [20, 100], 0),
    ("fp32", "fp32", 40, 2, 256, 192, 16, "heads", [130, 1], 64),
    ("fp32", "fp32", 3, 1, 20, 36, 3, "tokens", [130, 1], 0),
    ("bf16", "bf16", 32, 8, 128, 128, 16, "tokens", [5000, 1, 4097, 4096], 0),
    ("bf16", "int8", 8, 8, 32, 32, 128, "tokens", [3000, 2049], 2048),
    ("fp16", "e4m3", 64, 2, 64, 64, 16, "heads", [2500], 0),
    ("bf16", "bf16", 2, 2, 16, 16, 16, "tokens", [40, 9], 0),
    ("bf16", "bf16", 3, 3, 8, 24, 16, "heads", [40, 9], 0),
    ("bf16", "int8", 66, 2, 96, 96, 48, "heads", [700, 48, 95], 0),
]


def attention_case(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, seed=0, bad=(), pad=0):
    """A cache whose unused slots hold NaN, its table in no order, and the numbers each sequence sees."""
    t = T[dtype]
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + 3, max(need + [1]) + 1
    g = torch.Generator().manual_seed(seed)
    free = torch.randperm(pages, generator=g)
    cache, info = make_cache(dev, kind, order, pages, page, kv, dk, dv, pad)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    seen, at = [], 0
    slots_used = []
    for i, n in enumerate(need):
        table[i, :n] = free[at:at + n].int()
        at += n
        pos = torch.arange(lens[i])
        slots_used.append(table[i].long()[pos // page] * page + pos % page)
    total = pages * page
    sides = []
    for which, d in (("k", dk), ("v", dv)):
        x = torch.randn((total, kv, d), generator=g)
        s, ss = cache_strides(order, kv, page, d, pad)
        buf = getattr(cache, which)
        if kind in TOP:
            codes, scale = quantised64(x, kind)
            num = codes * scale.to(F64)[..., None]
            codes = codes.float().to(T[kind])
        else:
            codes, scale, num = x.to(t), None, x.to(t).to(F64)
        unused = torch.ones(total, dtype=torch.bool)
        for u in slots_used:
            unused[u] = False
        raw = torch.zeros(buf.numel(), dtype=codes.dtype)
        if kind not in TOP:
            codes[unused] = float("nan")
        raw.as_strided((pages, page, kv, d), s).copy_(codes.view(pages, page, kv, d))
        buf.copy_((raw.view(torch.uint8) if kind == "e4m3" else raw).to(dev))
        if scale is not None:
            scale[unused] = float("nan")
            getattr(cache, which + "_scale").as_strided((pages, page, kv), ss).copy_(scale.view(pages, page, kv).to(dev))
        sides.append(num)
    for i, col, val in bad:
        table[i, col] = val
    return cache, table, slots_used, sides


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,lens,window", ATTEND)
def test_attention(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, window):
    t, b = T[dtype], len(lens)
    cache, table, slots, (kn, vn) = attention_case(dev, dtype, kind, heads, kv, dk, dv, page, order, lens)
    q = rand((b, heads, dk), t, 11)
    out = torch.full((b, heads, dv), -7.0, dtype=t, device=dev)
    lse = torch.full((b, heads), -7.0, device=dev)
    Lq, Lo = f"({dk},{heads},{b}):(1,{dk},{heads * dk})", f"({dv},{heads},{b}):(1,{dv},{heads * dv})"
    args = (q.to(dev), Lq, cache, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev))
    lr.paged_attention(*args, out, Lo, window=window, lse=lse)
    seen = [u[max(0, len(u) - window):] if window else u for u in slots]
    want, wlse, tol = attention64(q, [kn[u] for u in seen], [vn[u] for u in seen], dk ** -0.5, t, kind)
    close(out, want, tol, "out")
    close(lse, wlse, tol.lse, "lse")
    again = torch.empty_like(out)
    lr.paged_attention(*args, again, Lo, window=window)
    assert torch.equal(out, again)                # the same bits every time, with or without lse


def test_attention_bad_pages_and_lengths(dev):
    """Tokens of a page outside the cache are left out; lengths below zero and past the table are limited."""
    for dtype, kind in (("bf16", "bf16"), ("fp16", "e4m3"), ("fp32", "fp32")):
        lens = [100, 100, 40, 64]
        bad = [(0, 1, -1), (0, 3, 1 << 30), (1, 0, -5), (2, 0, 99999), (2, 1, -1), (2, 2, -2 ** 31)]
        cache, table, slots, (kn, vn) = attention_case(dev, dtype, kind, 8, 2, 64, 64, 16, "tokens", lens, bad=bad)
        t = T[dtype]
        q = rand((4, 8, 64), t, 2)
        out, lse = torch.empty((4, 8, 64), dtype=t, device=dev), torch.empty((4, 8), device=dev)
        L = "(64,8,4):(1,64,512)"
        width = 4                                   # pages the table has for this call: 64 tokens
        given = torch.tensor([100, 2 ** 31 - 1, 40, -3], dtype=torch.int32, device=dev)
        lr.paged_attention(q.to(dev), L, cache, table.to(dev)[:, :width], given, out, L, lse=lse)
        ok = {0: [0, 2], 1: [1, 2, 3], 2: [], 3: []}
        seen = [torch.cat([slots[i][c * 16:c * 16 + 16] for c in ok[i]]) if ok[i] else slots[i][:0] for i in range(4)]
        want, wlse, tol = attention64(q, [kn[u] for u in seen], [vn[u] for u in seen], 0.125, t, kind)
        close(out, want, tol)
        close(lse, wlse, tol.lse)
        assert (out[2:] == 0).all() and (lse[2:] == -math.inf).all()


@pytest.mark.parametrize("dtype,kind", [("bf16", "bf16"), ("fp16", "int8"), ("fp32", "fp32")])
def test_attention_strides(dev, dtype, kind):
    """Padded cache rows, q and out in another order, a part of the sequences, buffers off 16 bytes."""
    t, heads, kv, d, lens = T[dtype], 4, 2, 64, [90, 33, 17]
    for pad, off in ((16, 0), (3, 1)):
        cache, table, slots, (kn, vn) = attention_case(dev, dtype, kind, heads, kv, d, d, 16, "heads", lens, pad=pad)
        b = len(lens)
        q = rand((b, heads, d), t, 4)
        qb = torch.zeros(heads * b * (d + 8) + off, dtype=t)
        qb[off:].as_strided((b, heads, d), (d + 8, b * (d + 8), 1)).copy_(q)
        ob = torch.full((heads * b * d + off,), -7.0, dtype=t, device=dev)
        Lq = f"({d},{heads},{b}):(1,{b * (d + 8)},{d + 8})"
        Lo = f"({d},{heads},{b}):({heads * b},{b},1)"
        lr.paged_attention(qb.to(dev)[off:], Lq, cache, table.to(dev), torch.tensor(lens[:2], dtype=torch.int32, device=dev),
                           ob[off:], Lo, scale=0.3)
        got = ob.cpu()[off:].as_strided((b, heads, d), (1, b, heads * b))
        want, _, tol = attention64(q[:2], [kn[u] for u in slots[:2]], [vn[u] for u in slots[:2]], 0.3, t, kind)
        close(got[:2], want, tol)
        assert (got[2] == -7).all()


def test_attention_large_scores(dev):
    """Scores far apart: one key takes all, sums stay finite; and equal scores give the mean."""
    for dtype, kind in (("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32")):
        t = T[dtype]
        cache, table, slots, (kn, vn) = attention_case(dev, dtype, kind, 2, 1, 64, 64, 16, "tokens", [200])
        q = rand((1, 2, 64), t, 6) * 50
        q[0, 1] = 0
        out, lse = torch.empty((1, 2, 64), dtype=t, device=dev), torch.empty((1, 2), device=dev)
        L = "(64,2,1):(1,64,128)"
        lr.paged_attention(q.to(dev), L, cache, table.to(dev), torch.tensor([200], dtype=torch.int32, device=dev), out, L,
                           scale=4.0, lse=lse)
        want, wlse, tol = attention64(q, [kn[slots[0]]], [vn[slots[0]]], 4.0, t, kind)
        close(out, want, tol)
        close(lse, wlse, tol.lse)


def test_side_stream_and_graph(dev):
    """One decoding step (rotate the query, store the token, attend) on another stream, then captured into a
    graph and replayed with new inputs, against the same calls made eagerly."""
    b, h, kv, d, page, width = 3, 8, 2, 64, 16, 40
    pages = b * width
    g = torch.Generator().manual_seed(5)
    table = torch.randperm(pages, generator=g).int().view(b, width).to(dev)
    rt = lr.rope_table(d, device=dev)
    L, Lk = lr.Layout(f"({d},{h},{b}):(1,{d},{h * d})"), lr.Layout(f"({d},{kv},{b}):(1,{d},{kv * d})")

    def fresh():
        k, v = (torch.zeros(pages * page * kv * d, dtype=torch.uint8, device=dev) for _ in range(2))
        ks, vs = (torch.zeros(pages * page * kv, device=dev) for _ in range(2))
        lay = f"({d},{kv},{page},{pages}):(1,{d},{kv * d},{page * kv * d})"
        return lr.PagedCache(k, lay, v, lay, ks, vs, f"({kv},{page},{pages}):(1,{kv},{page * kv})")

    def inputs(i):
        pos = torch.tensor([i, 200 + i, 500 + i], device=dev)
        q, k, v = (rand((b, n, d), torch.bfloat16, 100 * i + n + j).to(dev) for j, n in enumerate((h, kv, kv)))
        slots = table.long()[torch.arange(b, device=dev), pos // page] * page + pos % page
        return q, k, v, pos, slots, (pos + 1).int()

    def step(cache, x, qr, out, ws, stream=None):
        q, k, v, pos, slots, lens = x
        lr.rope(q, L, qr, L, pos, rt, stream=stream)
        lr.cache_write(cache, k, Lk, v, Lk, slots, table=rt, positions=pos, stream=stream)
        lr.paged_attention(qr, L, cache, table, lens, out, L, workspace=ws, stream=stream)

    need = lr.paged_attention_plan(L, fresh(), L, width, torch.bfloat16)["workspace_bytes"]
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    eager, want = fresh(), []
    for i in range(6):
        out, qr = (torch.empty((b, h, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
        step(eager, inputs(i), qr, out, ws)
        want.append(out)
    torch.cuda.synchronize()
    # another stream, workspace allocated by the call
    side, cache = torch.cuda.Stream(), fresh()
    xs = [inputs(i) for i in range(6)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        out, qr = (torch.empty((b, h, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
        torch.cuda.synchronize()
        step(cache, xs[i], qr, out, None, stream=side)
        got.append(out)
        side.synchronize()
    assert all(torch.equal(a, w) for a, w in zip(got, want))
    # a graph, its inputs copied in before each replay
    cache, x = fresh(), [z.clone() for z in xs[0]]
    out, qr = (torch.empty((b, h, d), dtype=torch.bfloat16, device=dev) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, x, qr, out, ws)
    for i in range(6):
        for dst, src in zip(x, xs[i]):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
        torch.randn(1 << 20, device=dev).sum().item()    # eager work between the replays


# ------------------------------------------------------------------------------------ splits, chunks and codes
ATTEND_RUNS = [  # type, kind, heads, kv, dk, dv, page, order, lens, window: many sequences, many parts, ragged chunks
    ("bf16", "e4m3", 4, 2, 72, 72, 16, "heads", [40, 300, 5], 0),
    ("fp16", "int8", 4, 1, 24, 40, 16, "tokens", [40, 300, 5], 0),
    ("bf16", "int8", 2, 1, 16, 8, 16, "tokens", [700], 0),
    ("bf16", "e4m3", 3, 1, 8, 8, 16, "tokens", [70], 0),
    ("fp32", "e4m3", 34, 1, 72, 128, 16, "heads", [1300, 2], 0),
    ("fp32", "int8", 8, 4, 256, 200, 8, "tokens", [700, 0, 31], 300),
    ("fp32", "e4m3", 2, 1, 64, 64, 32, "tokens", [20000], 0),
    ("bf16", "bf16", 2, 1, 32, 32, 64, "tokens", [40000], 0),                            # over 64 parts of one sequence
    ("bf16", "bf16", 2, 1, 18, 32, 64, "tokens", [20000], 0),                            # the same, one key a lane
    ("bf16", "bf16", 2, 1, 32, 32, 16, "heads", [(i * 389) % 1500 for i in range(70)], 0),  # over 64 sequences, some empty
    ("fp16", "int8", 6, 2, 32, 64, 16, "heads", [(i * 977) % 900 for i in range(150)], 500),
    ("fp32", "fp32", 3, 3, 20, 20, 16, "heads", [(i * 389) % 1500 for i in range(67)], 0),
    ("fp32", "fp32", 3, 3, 18, 21, 16, "heads", [(i * 389) % 700 for i in range(67)], 0),
    ("bf16", "bf16", 1, 1, 64, 64, 16, "tokens", [0, 0, 6000, 0, 1, 0], 0),
    ("bf16", "e4m3", 40, 1, 128, 128, 16, "tokens", [3000, 10, 2000], 777),
]


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,lens,window", ATTEND_RUNS)
def test_attention_runs(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, window):
    test_attention(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, window)


def test_attention_uneven_batch_is_its_parts(dev):
    """How a sequence is cut depends on the others in the batch: alone or among others it stays within the tolerance
    of both, and the empty ones give zeros."""
    lens = [0, 7000, 1, 129, 0, 128]
    cache, table, slots, (kn, vn) = attention_case(dev, "bf16", "bf16", 8, 2, 128, 128, 16, "heads", lens)
    q = rand((6, 8, 128), torch.bfloat16, 3)
    want, wlse, tol = attention64(q, [kn[u] for u in slots], [vn[u] for u in slots], 128 ** -0.5, torch.bfloat16, "bf16")
    for first in (0, 1, 3):
        b = 6 - first
        L = f"(128,8,{b}):(1,128,1024)"
        out, lse = torch.full((b, 8, 128), -7.0, dtype=torch.bfloat16, device=dev), torch.full((b, 8), -7.0, device=dev)
        lr.paged_attention(q[first:].contiguous().to(dev), L, cache, table[first:].contiguous().to(dev),
                           torch.tensor(lens[first:], dtype=torch.int32, device=dev), out, L, lse=lse)
        close(out, want[first:], tol[first:])
        close(lse, wlse[first:], tol.lse[first:])


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_codes_at_ties(dev, dtype, kind):
    """Quotients on a tie and next to one, on either side, in rows whose scale is exact and in rows whose scale is
    rounded: simple parts of the row's largest value, and for fp32 their neighbours."""
    t, n, d = T[dtype], 200, 128
    g = torch.Generator().manual_seed(4)
    top = torch.randint(1, 256, (n, 1), generator=g).float()                  # 8 bits: exact in every type
    top[:40] = torch.tensor([7.0, 127.0, 112.0, 254.0] * 10)[:, None]         # scales without rounding
    part = torch.randint(0, 257, (n, d), generator=g).float() / 256 if kind == "e4m3" else \
        torch.randint(0, 255, (n, d), generator=g).float() / 254
    x = (top * part * (torch.randint(0, 2, (n, d), generator=g) * 2 - 1)).to(t)
    small = torch.randint(0, 2, (n, d), generator=g).bool() & (torch.arange(d) >= d // 2)
    x = torch.where(small, x * 2.0 ** -7, x)                                  # e4m3's smallest codes
    if dtype == "fp32":
        step = torch.randint(-2, 3, (n, d), generator=g, dtype=torch.int32)
        x = torch.where(x == 0, x, (x.view(torch.int32) + step).view(torch.float32))
        x = torch.minimum(x, top).maximum(-top)
    x[:, 0] = top[:, 0].to(t)
    x = x.reshape(n, 1, d).contiguous()
    cache, info = make_cache(dev, kind, "tokens", n, 1, 1, d, d)
    L = f"({d},1,{n}):(1,{d},{d})"
    slots = torch.arange(n)
    lr.cache_write(cache, x.to(dev), L, x.to(dev), L, slots.to(dev))
    codes, scale = quantised64(x, kind)
    for which in "kv":
        got, s = content(cache, info, d, which)
        close(s, scale.to(F64), 0.0)
        close(got, codes, 0.0, which)


def test_large_calls_stream(dev):
    """Calls past 256 MiB take streaming loads and stores: the same bits as in pieces that do not."""
    n, h, d = 12000, 48, 128
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn((n, h, d), generator=g, device=dev).to(torch.bfloat16)
    L = f"({d},{h},{n}):(1,{d},{h * d})"
    pos = torch.arange(n, device=dev)
    table = lr.rope_table(d, device=dev)
    y = lr.rope(x, L, torch.empty_like(x), L, pos, table)
    piece = 1000
    Lp = f"({d},{h},{piece}):(1,{d},{h * d})"
    for i in range(0, n, piece):
        z = lr.rope(x[i:i + piece], Lp, torch.empty_like(x[:piece]), Lp, pos[i:i + piece].contiguous(), table)
        assert torch.equal(z, y[i:i + piece]), i
    del y
    page = 16
    lay = f"({d},{h},{page},{n // page}):(1,{d},{h * d},{page * h * d})"

    def fresh():
        k, v = (torch.zeros(n * h * d, dtype=torch.int8, device=dev) for _ in range(2))
        ks, vs = (torch.zeros(n * h, device=dev) for _ in range(2))
        return lr.PagedCache(k, lay, v, lay, ks, vs, f"({h},{page},{n // page}):(1,{h},{page * h})")
    slots = torch.randperm(n, generator=g, device=dev)
    whole, parts = fresh(), fresh()
    lr.cache_write(whole, x, L, x, L, slots, table=table, positions=pos)
    for i in range(0, n, piece):
        lr.cache_write(parts, x[i:i + piece], Lp, x[i:i + piece], Lp, slots[i:i + piece].contiguous(), table=table,
                       positions=pos[i:i + piece].contiguous())
    assert torch.equal(whole.k, parts.k) and torch.equal(whole.v, parts.v)
    assert torch.equal(whole.k_scale, parts.k_scale) and torch.equal(whole.v_scale, parts.v_scale)
    a, b = lr.cache_read(whole, slots, torch.empty_like(x), L, torch.empty_like(x), L)
    c, e = (torch.empty((piece, h, d), dtype=x.dtype, device=dev) for _ in range(2))
    for i in range(0, n, piece):
        lr.cache_read(parts, slots[i:i + piece].contiguous(), c, Lp, e, Lp)
        assert torch.equal(a[i:i + piece], c) and torch.equal(b[i:i + piece], e), i


def test_rope_modes_of_many_leaves(dev):
    """Heads and tokens of three leaves each, which the chunked kernel does not take."""
    x = rand((2, 3, 2, 2, 2, 3, 16), torch.bfloat16, 8)             # tokens c, b, a; heads c, b, a; elements
    s = [1]
    for extent in reversed(x.shape[1:]):
        s.insert(0, s[0] * extent)
    perm = (1, 0, 2, 4, 3, 5, 6)                                     # of y's storage: neighbours that do not merge
    yshape = [x.shape[i] for i in perm]
    ys = [1]
    for extent in reversed(yshape[1:]):
        ys.insert(0, ys[0] * extent)
    at = {p: ys[i] for i, p in enumerate(perm)}
    Lx = f"(16,(3,2,2),(2,3,2)):(1,({s[5]},{s[4]},{s[3]}),({s[2]},{s[1]},{s[0]}))"
    Ly = f"(16,(3,2,2),(2,3,2)):(1,({at[5]},{at[4]},{at[3]}),({at[2]},{at[1]},{at[0]}))"
    pos = torch.arange(12) * 77
    table = lr.rope_table(16, device=dev)
    y = torch.full((x.numel(),), -7.0, dtype=x.dtype, device=dev)
    lr.rope(x.to(dev), Lx, y, Ly, pos.to(dev), table)
    # token index: a fastest; head index: a fastest
    want, size = rotate64(x.reshape(12, 12, 16), pos, table, "half")
    got = y.cpu().view(yshape).permute([perm.index(i) for i in range(7)]).reshape(12, 12, 16)
    close(got, want, rope_tolerance(want, size, torch.bfloat16))


@pytest.mark.parametrize("kw", [dict(), dict(cache="bf16", heads=4, kv_heads=4, dim=64, window=33),
                                dict(cache="int8", heads=20, kv_heads=1, dim=80, prompt=300)])
def test_decode_example(dev, kw):
    """The example's steps, each within its tolerance."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode.py")
    spec = importlib.util.spec_from_file_location("decode_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    args = dict(batch=3, heads=8, kv_heads=2, dim=128, prompt=150, steps=5, check=True)
    args.update(kw)
    _, out, worst = example.run(**args)
    assert out.isfinite().all() and worst <= 1


UNEVEN = [(i * 389) % 2000 for i in range(40)]
ATTEND_WIDE = [  # enough work for four cache heads a workgroup, where a token's heads lie next to each other; and
    # heads of 160 and 192, which have kernels of their own
    ("bf16", "bf16", 16, 4, 128, 128, 16, "tokens", UNEVEN, 0),
    ("fp16", "int8", 80, 4, 72, 72, 16, "tokens", UNEVEN, 0),
    ("bf16", "e4m3", 8, 8, 80, 64, 32, "tokens", UNEVEN[:25], 700),
    ("fp32", "fp32", 4, 4, 64, 96, 1, "tokens", UNEVEN, 0),
    ("fp16", "fp16", 24, 12, 32, 32, 7, "tokens", UNEVEN[:20], 0),
    ("fp32", "e4m3", 8, 4, 128, 128, 16, "tokens", UNEVEN, 0),
    ("bf16", "bf16", 4, 4, 160, 192, 16, "tokens", UNEVEN, 0),
    ("bf16", "bf16", 8, 4, 160, 160, 16, "heads", [700, 0, 31], 0),
    ("fp16", "int8", 3, 3, 192, 160, 16, "tokens", [700, 0, 31], 0),
    ("fp32", "fp32", 2, 2, 192, 136, 16, "heads", [300, 5], 0),
    ("bf16", "e4m3", 4, 4, 256, 256, 16, "tokens", UNEVEN, 0),
]


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,lens,window", ATTEND_WIDE)
def test_attention_wide(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, window):
    test_attention(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, window)


ATTEND_NARROW = [  # heads of up to 32, of 96 and of 160 beside the tests above: many query heads, four cache heads a workgroup
    ("fp32", "fp32", 20, 1, 32, 32, 16, "heads", [700, 0, 31], 0),
    ("bf16", "bf16", 40, 2, 24, 32, 16, "tokens", [700, 0, 31], 50),
    ("fp16", "fp16", 3, 3, 8, 8, 5, "heads", [1300, 2, 16], 0),
    ("fp32", "fp32", 4, 4, 4, 28, 16, "tokens", UNEVEN, 0),
    ("bf16", "bf16", 80, 4, 16, 32, 16, "tokens", UNEVEN, 0),
    ("bf16", "bf16", 20, 1, 72, 96, 16, "heads", [700, 0, 31], 0),
    ("fp32", "fp32", 20, 1, 96, 68, 16, "heads", [700, 0, 31], 0),
    ("fp16", "fp16", 20, 1, 136, 160, 16, "heads", [700, 0, 31], 0),
]


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,lens,window", ATTEND_NARROW)
def test_attention_narrow(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, window):
    test_attention(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, window)


def test_attention_wide_plan_off_alignment(dev):
    """A plan for four heads a workgroup whose buffers turn out to be off 16 bytes: one key a lane instead, with the
    same workspace."""
    heads, kv, d, page, lens = 8, 4, 64, 16, UNEVEN
    cache, table, slots, (kn, vn) = attention_case(dev, "bf16", "bf16", heads, kv, d, d, page, "tokens", lens)
    pages = cache.k.numel() // (page * kv * d)
    lay = f"({d},{kv},{page},{pages}):(1,{d},{kv * d},{page * kv * d})"
    off = [torch.cat([t.new_zeros(1), t])[1:] for t in (cache.k, cache.v)]
    assert off[0].data_ptr() % 16 == 2
    moved = lr.PagedCache(off[0], lay, off[1], lay)
    q = rand((len(lens), heads, d), torch.bfloat16, 3)
    L = f"({d},{heads},{len(lens)}):(1,{d},{heads * d})"
    out, lse = torch.empty((len(lens), heads, d), dtype=torch.bfloat16, device=dev), torch.empty((len(lens), heads), device=dev)
    lr.paged_attention(q.to(dev), L, moved, table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), out, L, lse=lse)
    want, wlse, tol = attention64(q, [kn[u] for u in slots], [vn[u] for u in slots], d ** -0.5, torch.bfloat16, "bf16")
    close(out, want, tol)
    close(lse, wlse, tol.lse)


# ------------------------------------------------------------------------------------ NaN, infinities, small numbers
QUIET = {"fp32": [0x7fffffff, 0xffffffff, 0x7ffffffc, 0xfffffffc, 0x7fc00000], "fp16": [0x7fff, 0xffff, 0x7e00],
         "bf16": [0x7fff, 0xffff, 0x7fc0]}


def put_bits(x, at, dtype, bits):
    """x with the bit patterns `bits` at the flat places `at`."""
    whole = torch.int32 if dtype == "fp32" else torch.int16
    top = 1 << (32 if whole == torch.int32 else 16)
    pattern = torch.tensor([b - top if b >= top // 2 else b for b in bits], dtype=whole)
    x.view(whole).view(-1)[at] = pattern
    return x


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("d", [128, 72, 33])
def test_cache_write_nan(dev, dtype, kind, d, patterns=QUIET):
    """NaN of every payload, all ones among them, at every place of a row: it stays NaN in e4m3 and becomes 0 in
    int8, and neither the scale nor the other codes of its row notice."""
    t, n = T[dtype], 4 * d
    k, v = rand((n, 1, d), t, 1), rand((n, 1, d), t, 2)
    bits = patterns[dtype]
    rows = torch.arange(n)
    for x, first in ((k, 0), (v, 3)):
        put_bits(x, rows * d + rows % d, dtype, [bits[(int(i) // 2 + first) % len(bits)] for i in rows])
        assert int(x.isnan().sum()) == n
    cache, info = make_cache(dev, kind, "tokens", n, 1, 1, d, d)
    L = f"({d},1,{n}):(1,{d},{d})"
    lr.cache_write(cache, k.to(dev), L, v.to(dev), L, torch.arange(n).to(dev))
    for x, which in ((k, "k"), (v, "v")):
        codes, scale = quantised64(x, kind)
        got, s = content(cache, info, d, which)
        close(s, scale.to(F64), 0.0, which + " scales")
        close(got, codes, 0.0, which)


SIGNALLING = {"fp32": [0x7f800001, 0xff800001, 0x7fbfffff], "fp16": [0x7c01, 0xfdff], "bf16": [0x7f81, 0xffbf]}


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("d", [128, 72, 33])
def test_cache_write_signalling_nan(dev, dtype, kind, d):
    """The same of signalling NaN, which some instructions answer with a NaN where they pass over a quiet one."""
    test_cache_write_nan(dev, dtype, kind, d, SIGNALLING)


# Forms of the attention: one run a head or several, heads side by side, one key a lane, up to 32 query heads a workgroup.
FORMS = [  # heads, kv, dk, dv, page, order, lens
    (4, 2, 64, 64, 16, "tokens", [40, 300]),
    (2, 1, 64, 64, 16, "heads", [2500, 7]),
    (16, 4, 128, 128, 16, "tokens", [(i * 389) % 2000 + 1 for i in range(40)]),
    (20, 1, 72, 96, 16, "heads", [700, 33]),
    (2, 1, 160, 160, 16, "heads", [700, 33]),
    (3, 3, 33, 17, 5, "tokens", [1200, 4]),
]


def attend_all(dev, cache, table, q, dv, lens, **kw):
    """(out, lse) of one call, q (sequences, heads, dk) on the CPU."""
    b, h, dk = q.shape
    out = torch.full((b, h, dv), -7.0, dtype=q.dtype, device=dev)
    lse = torch.full((b, h), -7.0, device=dev)
    lr.paged_attention(q.to(dev), f"({dk},{h},{b}):(1,{dk},{h * dk})", cache, table.to(dev),
                       torch.tensor(lens, dtype=torch.int32, device=dev), out, f"({dv},{h},{b}):(1,{dv},{h * dv})", lse=lse, **kw)
    return out, lse


def set_rows(cache, which, order, page, kv, d, slots, rows):
    """The cache's rows of the given slots: rows (len(slots), kv, d)."""
    buf = getattr(cache, which)
    s, _ = cache_strides(order, kv, page, d)
    pages = (buf.numel() - 1) // s[0] + 1
    view = buf.as_strided((pages, page, kv, d), s)
    view[(slots // page).to(buf.device), (slots % page).to(buf.device)] = rows.to(buf.dtype).to(buf.device)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("heads,kv,dk,dv,page,order,lens", FORMS)
def test_attention_infinite_values(dev, dtype, heads, kv, dk, dv, page, order, lens):
    """An infinite value makes its column infinite, two of different signs or a NaN make it NaN, and no other column
    notices; infinities that are not seen do not matter."""
    t, b = T[dtype], len(lens)
    cache, table, slots, (kn, vn) = attention_case(dev, dtype, dtype, heads, kv, dk, dv, page, order, lens)
    q = rand((b, heads, dk), t, 11)
    for i, u in enumerate(slots):
        n = len(u)
        for column, row, value in ((0, 0, math.inf), (1, n - 1, -math.inf), (2, n // 2, math.inf), (3, n // 3, math.nan)):
            vn[u[row], :, column] = value
        if n > 1:
            vn[u[0], :, 5], vn[u[1], :, 5] = math.inf, -math.inf
            vn[u[0], :, 6], vn[u[n - 1], :, 6] = -math.inf, -math.inf
        set_rows(cache, "v", order, page, kv, dv, u, vn[u].to(t))
    out, lse = attend_all(dev, cache, table, q, dv, lens)
    finite = vn.nan_to_num(0, 0, 0)
    want, wlse, tol = attention64(q, [kn[u] for u in slots], [finite[u] for u in slots], dk ** -0.5, t, dtype)
    for i, u in enumerate(slots):
        for column in range(7):
            x = vn[u][:, :, column]
            bad = x.isnan().any() or ((x == math.inf).any() and (x == -math.inf).any())
            if bad or x.isinf().any():
                want[i, :, column] = math.nan if bad else x[x.isinf()].max()
    close(out, want, tol, "out")
    close(lse, wlse, tol.lse, "lse")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("d", [64, 33])
def test_attention_infinite_value_of_small_weight(dev, dtype, d):
    """The weight of an infinite value may be e^-30 of the largest."""
    t, n = T[dtype], 100
    cache, table, slots, (kn, vn) = attention_case(dev, dtype, dtype, 2, 1, d, d, 16, "heads", [n])
    u = slots[0]
    kn[u] = 0
    kn[u[::32], :, 0], vn[u[70], :, 1], vn[u[71], :, 2] = 30, math.inf, -math.inf
    set_rows(cache, "k", "heads", 16, 1, d, u, kn[u])
    set_rows(cache, "v", "heads", 16, 1, d, u, vn[u])
    q = torch.zeros((1, 2, d), dtype=t)
    q[..., 0] = 1
    out, _ = attend_all(dev, cache, table, q, d, [n], scale=1.0)
    want, _, tol = attention64(q, [kn[u]], [vn[u].nan_to_num(0, 0, 0)], 1.0, t, dtype)
    want[..., 1], want[..., 2] = math.inf, -math.inf
    close(out, want, tol)


@pytest.mark.parametrize("dtype,kind", [("bf16", "bf16"), ("fp16", "int8"), ("fp32", "fp32"), ("bf16", "e4m3")])
@pytest.mark.parametrize("heads,kv,dk,dv,page,order,lens", FORMS)
def test_attention_nan_query(dev, dtype, kind, heads, kv, dk, dv, page, order, lens):
    """A NaN in a head's query: its output and its lse are NaN, in one part or in several; other heads do not notice,
    and a sequence without tokens still has none."""
    t, lens = T[dtype], lens + [0]
    b = len(lens)
    cache, table, slots, (kn, vn) = attention_case(dev, dtype, kind, heads, kv, dk, dv, page, order, lens)
    q = rand((b, heads, dk), t, 11)
    clean = q.clone()
    for i in range(b):
        q[i, i % heads, (5 * i) % dk] = math.nan
    out, lse = attend_all(dev, cache, table, q, dv, lens)
    want, wlse, tol = attention64(clean, [kn[u] for u in slots], [vn[u] for u in slots], dk ** -0.5, t, kind)
    for i in range(b - 1):
        want[i, i % heads], wlse[i, i % heads] = math.nan, math.nan
    close(out, want, tol, "out")
    close(lse, wlse, tol.lse, "lse")


def tight64(q, ks, vs, scale, weight, floor):
    """attention64 with a tolerance without slack for the weights: `weight` relative to each and `floor` relative to
    the largest."""
    b, h, dk = q.shape
    dv = vs[0].shape[-1]
    out, tol = torch.zeros((b, h, dv), dtype=F64), torch.zeros((b, h, dv), dtype=F64)
    for i in range(b):
        g = h // ks[i].shape[1]
        k, v = (x[i].to(F64).repeat_interleave(g, 1).transpose(0, 1) for x in (ks, vs))
        s = torch.matmul(k, q[i].to(F64).unsqueeze(-1)).squeeze(-1) * scale
        p = torch.softmax(s, -1)
        out[i] = torch.matmul(p.unsqueeze(1), v).squeeze(1)
        size = torch.matmul(p.unsqueeze(1), v.abs()).squeeze(1)
        # a score: a rounding for each product of its row and for the scale; the exponential's own 2^-22
        ds = (torch.matmul(k.abs(), q[i].to(F64).abs().unsqueeze(-1)).squeeze(-1) * abs(scale)).amax(-1) * (dk + 8) * U
        lost = floor * p.amax(-1)[:, None] * v.abs().sum(1)
        tol[i] = HALF[q.dtype] * out[i].abs() + (weight + (k.shape[1] + 16) * U + 2 * ds[:, None] + 2.0 ** -22) * size + lost \
            + TINY[q.dtype]
    return out, tol


@pytest.mark.parametrize("heads,kv,dk,dv,page,order", [(2, 1, 64, 64, 16, "heads"), (8, 8, 64, 64, 16, "tokens"),
                                                       (20, 1, 64, 32, 16, "heads"), (1, 1, 160, 192, 16, "heads"),
                                                       (2, 2, 33, 20, 16, "tokens")])
@pytest.mark.parametrize("below", [10.0, 15.0, 16.0, 17.0, 17.8])
def test_attention_sinks_fp16(dev, heads, kv, dk, dv, page, order, below):
    """Tokens far above all others whose values are zero, one in every 32: what the others weigh is under 2^-21 of the
    largest weight, and they alone make up the output, which still has the accuracy of fp16."""
    n = 20000 if order == "heads" else 60000
    cache, table, slots, (kn, vn) = attention_case(dev, "fp16", "fp16", heads, kv, dk, dv, page, order, [n])
    u = slots[0]
    kn[u], vn[u] = 0, 1000 * (1 + rand((n, kv, dv), torch.float16, 3).abs().to(F64).clamp(max=4))
    kn[u[::32], :, 0], vn[u[::32]] = below, 0
    kn[u], vn[u] = kn[u].to(torch.float16).to(F64), vn[u].to(torch.float16).to(F64)
    for which, x, d in (("k", kn, dk), ("v", vn, dv)):
        set_rows(cache, which, order, page, kv, d, u, x[u])
    q = torch.zeros((1, heads, dk), dtype=torch.float16)
    q[..., 0] = 1
    out, _ = attend_all(dev, cache, table, q, dv, [n], scale=1.0)
    # two fp16 parts leave 2^-11 of 2^-11 of a weight, and at least half of 2^-24 where the largest is 2^7 or more
    want, tol = tight64(q, [kn[u]], [vn[u]], 1.0, 2.0 ** -22, 2.0 ** -32)
    close(out, want, tol)


@pytest.mark.parametrize("dtype,kind,weight,floor", [("bf16", "bf16", 2.0 ** -16, 0.0), ("fp16", "fp16", 2.0 ** -22, 2.0 ** -32),
                                                     ("fp16", "e4m3", 2.0 ** -16, 0.0), ("fp32", "fp32", 2.0 ** -24, 0.0)])
@pytest.mark.parametrize("heads,kv,dk,dv,page,order,lens", FORMS)
def test_attention_weights_in_two_parts(dev, dtype, kind, weight, floor, heads, kv, dk, dv, page, order, lens):
    """Values that nearly cancel, token by token, so that the output shows what the weights' rounding leaves: 16 bits
    of them (22 in fp16), as two parts have, not the 8 or 11 of one."""
    t, b = T[dtype], len(lens)
    cache, table, slots, (kn, vn) = attention_case(dev, dtype, kind, heads, kv, dk, dv, page, order, lens)
    for u in slots:
        m = len(u) // 2
        vn[u[m:2 * m]] = -vn[u[:m]]
        kn[u[m:2 * m]] = kn[u[:m]]
        if kind in TOP:       # codes: the scale of a key changes by a step or two, and its score with it
            for which, d in (("k", dk), ("v", dv)):
                s, ss = cache_strides(order, kv, page, d)
                buf, sc = getattr(cache, which), getattr(cache, which + "_scale")
                pages = sc.numel() // (page * kv)
                bv, sv = buf.as_strided((pages, page, kv, d), s), sc.as_strided((pages, page, kv), ss)
                a, z = u[:m].to(dev), u[m:2 * m].to(dev)
                bv[z // page, z % page] = bv[a // page, a % page]
                sign = 1 + 2.0 ** -7 if which == "k" else -1
                sv[z // page, z % page] = sv[a // page, a % page] * sign
            kn[u[m:2 * m]] = (kn[u[:m]] * (1 + 2.0 ** -7))
        else:
            kn[u[m:2 * m], :, 0] += 2.0 ** -5
            kn[u] = kn[u].to(t).to(F64)
            for which, x, d in (("k", kn, dk), ("v", vn, dv)):
                set_rows(cache, which, order, page, kv, d, u, x[u].to(t))
    q = rand((b, heads, dk), t, 11)
    out, _ = attend_all(dev, cache, table, q, dv, lens)
    want, tol = tight64(q, [kn[u] for u in slots], [vn[u] for u in slots], dk ** -0.5, weight, floor)
    close(out, want, tol)


@pytest.mark.parametrize("d", [256, 30])
def test_rope_small_angles(dev, d):
    """Sine and cosine of the slowest pairs and the first positions, relative to themselves: an angle has 32 bits
    however small it is.  Roundings: the angle's conversion, its constant and its product, and two in each series."""
    n = 40
    pos = torch.tensor([0, 1, 2, 3, 5, -1, -7] + [10 ** i for i in range(1, 7)] + list(range(100, 127)))[:n]
    table = lr.rope_table(d, base=1e8, device=dev)
    x = torch.zeros((n, 1, d))
    x[..., :d // 2] = 1
    L = f"({d},1,{n}):(1,{d},{d})"
    y = lr.rope(x.to(dev), L, torch.empty_like(x, device=dev), L, pos.to(dev), table).cpu().to(F64)
    a = (pos.reshape(-1, 1) * table.turns.cpu()).to(F64) * (2 * math.pi / 2.0 ** 64)
    cos, sin = y[:, 0, :d // 2], y[:, 0, d // 2:]
    close(sin, a.sin(), torch.where(a.abs() < math.pi / 4, 5 * U * a.sin().abs(), torch.full_like(a, 4 * U)), "sin")
    close(cos, a.cos(), 4 * U, "cos")


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [128, 33])
def test_codes_of_tiny_rows(dev, kind, d):
    """Rows whose scale is just above its least value, of numbers nearest to ties: what is left of a number after
    its tie has bits below fp32's smallest."""
    n = 64
    g = torch.Generator().manual_seed(4)
    scale = (1 + torch.randint(1, 1 << 23, (n, 1), generator=g).to(F64) / 2 ** 23) * 2.0 ** -126
    part = torch.randint(8, 16, (n, d), generator=g).to(F64) / 8 + 1 / 16 if kind == "e4m3" else \
        torch.randint(0, 2, (n, d), generator=g).to(F64) + 0.5
    sign = torch.randint(0, 2, (n, d), generator=g) * 2 - 1
    x = (scale * part * sign).float()
    x[:, 0] = (scale[:, 0] * TOP[kind]).float()
    x = x.reshape(n, 1, d).contiguous()
    cache, info = make_cache(dev, kind, "tokens", n, 1, 1, d, d)
    L = f"({d},1,{n}):(1,{d},{d})"
    lr.cache_write(cache, x.to(dev), L, x.to(dev), L, torch.arange(n).to(dev))
    codes, want = quantised64(x, kind)
    for which in "kv":
        got, s = content(cache, info, d, which)
        close(s, want.to(F64), 0.0, which + " scales")
        close(got, codes, 0.0, which)


def test_calls_of_nothing(dev):
    """No sequences, no tokens: empty tensors are taken, and nothing is written."""
    cache, table, slots, _ = attention_case(dev, "bf16", "bf16", 4, 2, 64, 64, 16, "tokens", [40, 300])
    kept = cache.k.clone()
    q = rand((2, 4, 64), torch.bfloat16, 1).to(dev)
    out, lse = torch.full((2, 4, 64), -7.0, dtype=torch.bfloat16, device=dev), torch.empty((0, 4), device=dev)
    L = "(64,4,2):(1,64,256)"
    none = torch.empty(0, dtype=torch.int32, device=dev)
    lr.paged_attention(q, L, cache, table.to(dev)[:0], none, out, L, lse=lse)
    lr.paged_attention(q, L, cache, table.to(dev), none, out, L)
    x = rand((2, 2, 64), torch.bfloat16, 2).to(dev)
    Lx, none = "(64,2,2):(1,64,128)", torch.empty(0, dtype=torch.int64, device=dev)
    rt = lr.rope_table(64, device=dev)
    lr.cache_write(cache, x, Lx, x, Lx, none, table=rt, positions=none)
    y, z = torch.full_like(x, -7.0), torch.full_like(x, -7.0)
    lr.cache_read(cache, none, y, Lx, z, Lx)
    lr.rope(x, Lx, y, Lx, none, rt)
    torch.cuda.synchronize()
    assert (out == -7).all() and (y == -7).all() and (z == -7).all()
    assert torch.equal(cache.k.view(torch.int16), kept.view(torch.int16))


def test_attention_table_of_one_page(dev):
    """A table of one page a sequence has contiguous rows whatever its second stride says."""
    lens = [3, 16, 9]
    cache, table, slots, (kn, vn) = attention_case(dev, "bf16", "bf16", 4, 2, 64, 64, 16, "tokens", lens)
    q = rand((3, 4, 64), torch.bfloat16, 1)
    column = table[:, 0].contiguous().view(1, 3).t()
    assert column.shape == (3, 1) and column.stride(1) != 1
    out, lse = attend_all(dev, cache, column, q, 64, lens)
    want, wlse, tol = attention64(q, [kn[u] for u in slots], [vn[u] for u in slots], 0.125, torch.bfloat16, "bf16")
    close(out, want, tol)
    close(lse, wlse, tol.lse)


WIDE_TABLES = [  # type, kind, heads, kv, dk, dv, page, order, lens, pages of the table, window
    ("bf16", "bf16", 32, 8, 128, 128, 16, "tokens", [1000] * 64, 8192, 0),
    ("bf16", "bf16", 32, 8, 128, 128, 16, "heads", [(i * 389) % 4097 for i in range(32)], 8192, 0),
    ("fp16", "int8", 8, 2, 64, 64, 16, "heads", [(i * 389) % 900 for i in range(150)], 4096, 0),
    ("fp32", "fp32", 8, 4, 64, 64, 16, "tokens", [(i * 389) % 900 for i in range(80)], 4096, 0),
    ("bf16", "e4m3", 8, 8, 128, 128, 16, "tokens", [5000, 0, 1, 4999] * 10, 8192, 4000),
    ("bf16", "bf16", 12, 3, 33, 17, 16, "tokens", [(i * 389) % 1200 for i in range(70)], 8192, 0),
]


@pytest.mark.parametrize("dtype,kind,heads,kv,dk,dv,page,order,lens,width,window", WIDE_TABLES)
def test_attention_wide_tables(dev, dtype, kind, heads, kv, dk, dv, page, order, lens, width, window):
    """Lengths far below the table's width: a run is then several blocks at least, the parts stay inside the
    workspace, and what lies behind it stays as it was."""
    t, b = T[dtype], len(lens)
    cache, table, slots, (kn, vn) = attention_case(dev, dtype, kind, heads, kv, dk, dv, page, order, lens)
    wide = torch.full((b, width), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    q = rand((b, heads, dk), t, 11)
    need = lr.paged_attention_plan(f"({dk},{heads},{b}):(1,{dk},{heads * dk})", cache, f"({dv},{heads},{b}):(1,{dv},{heads * dv})",
                                   width, t, window=window)
    assert need["splits"] > 1
    workspace = torch.full((need["workspace_bytes"] + 4096,), 0x5a, dtype=torch.uint8, device=dev)
    out, lse = attend_all(dev, cache, wide, q, dv, lens, window=window, workspace=workspace)
    seen = [u[max(0, len(u) - window):] if window else u for u in slots]
    want, wlse, tol = attention64(q, [kn[u] for u in seen], [vn[u] for u in seen], dk ** -0.5, t, kind)
    close(out, want, tol, "out")
    close(lse, wlse, tol.lse, "lse")
    assert (workspace[need["workspace_bytes"]:] == 0x5a).all()
