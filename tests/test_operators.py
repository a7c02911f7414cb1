"""Host side of the attention operators (no GPU): the frequency table, the plan, and every refusal.

Refusals are checked before anything is launched, so made-up pointers do: nothing is read through them.
"""

import ctypes
import math
import random

import pytest

import layout_remapping_copy_amd as lr
from layout_remapping_copy_amd import binding as B

torch = pytest.importorskip("torch")


def table(rot, **kw):
    t = lr.rope_table(rot, device="cpu", **kw)
    return [int(x) % 2 ** 64 / 2 ** 64 for x in t.turns], t.magnitude


@pytest.mark.parametrize("rot", [2, 16, 96, 128, 1024])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
def test_frequencies(rot, base):
    got, m = table(rot, base=base)
    assert m == 1.0 and len(got) == rot // 2
    for i, f in enumerate(got):
        want = base ** (-2.0 * i / rot) / (2 * math.pi)
        assert abs(f - want) <= 2.0 ** -50 * want + 2.0 ** -63   # the double on the right: a few steps of 2^-53


def test_scaled_frequencies():
    rot, base, factor, length = 64, 10000.0, 8.0, 4096.0
    plain, _ = table(rot, base=base)
    for a, b in zip(plain, table(rot, base=base, scaling="linear", factor=factor)[0]):
        assert abs(b - a / factor) <= 2.0 ** -60
    for a, b in zip(table(rot, base=base * factor ** (rot / (rot - 2)))[0],
                    table(rot, base=base, scaling="base", factor=factor)[0]):
        assert abs(a - b) <= 2.0 ** -48
    # by parts: fast pairs keep their frequency, slow ones are stretched, a ramp between
    got, m = table(rot, base=base, scaling="parts", factor=factor, original_len=length, low=1.0, high=32.0)
    assert abs(m - (0.1 * math.log(factor) + 1)) < 1e-15

    def at(times):
        return rot * math.log(length / (times * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = math.floor(at(32.0)), math.ceil(at(1.0))
    for i, (a, b) in enumerate(zip(plain, got)):
        keep = 1 - min(max((i - lo) / (hi - lo), 0), 1)
        assert abs(b - (a / factor * (1 - keep) + a * keep)) <= 2.0 ** -50
    assert got[0] == plain[0] and abs(got[-1] - plain[-1] / factor) <= 2.0 ** -60
    # by bands of the turns over the original length
    got, m = table(rot, base=base, scaling="bands", factor=factor, original_len=length, low=1.0, high=4.0)
    assert m == 1.0
    for a, b in zip(plain, got):
        keep = min(max((length * a - 1.0) / 3.0, 0), 1)
        assert abs(b - (a / factor * (1 - keep) + a * keep)) <= 2.0 ** -50


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=3), dict(rot=1026), dict(rot=-2), dict(base=1.0), dict(base=math.nan),
                                dict(base=math.inf), dict(scaling="linear", factor=0.0),
                                dict(scaling="linear", factor=math.nan), dict(scaling="parts", factor=2.0),
                                dict(scaling="bands", factor=2.0, original_len=10.0, low=4.0, high=4.0),
                                dict(scaling="bands", factor=2.0, original_len=10.0, low=0.0, high=4.0),
                                dict(scaling="base", factor=1e-9, base=2.0)])
def test_frequency_refusals(kw):
    kw = dict(kw)
    with pytest.raises(lr.LayoutRemapError) as e:
        lr.rope_table(kw.pop("rot", 64), device="cpu", **kw)
    assert e.value.code == B.ERR_INVALID
    assert lr.lib().lr_rope_table(None, None, None) == B.ERR_INVALID


def test_frequency_names():
    with pytest.raises(ValueError):
        lr.rope_table(64, scaling="twice", device="cpu")


# -------------------------------------------------------------------------------- refusals
X, Y, V, W, S = 0x100000, 0x40000000, 0x80000000, 0xc0000000, 0x200000  # far apart, never read


def rope(**kw):
    a = dict(x=X, Lx="(64,4,10):(1,64,256)", cx=2560, y=Y, Ly="(64,4,10):(1,64,256)", cy=2560, dtype=B.BF16,
             turns=S, positions=S, rot=64, pairs=0, Lp=None, cp=10, n=10, flags=0)
    a.update(kw)
    lay = {k: (lr.Layout(a[k]).c if a[k] is not None else None) for k in ("Lx", "Ly", "Lp")}
    r = B.lr_rotation(a["turns"], a["positions"], a["rot"], a["pairs"], 1.0) if a["rot"] is not None else None
    return lr.lib().lr_rope(a["x"], lay["Lx"], a["cx"], a["y"], lay["Ly"], a["cy"], a["dtype"], r, lay["Lp"], a["cp"],
                            a["n"], a["flags"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), B.ERR_INVALID), (dict(y=None), B.ERR_INVALID), (dict(Lx=None), B.ERR_INVALID),
    (dict(rot=None), B.ERR_INVALID), (dict(turns=None), B.ERR_INVALID), (dict(positions=None), B.ERR_INVALID),
    (dict(dtype=B.E4M3), B.ERR_TYPE), (dict(dtype=9), B.ERR_TYPE), (dict(dtype=-1), B.ERR_TYPE),
    (dict(rot=66), B.ERR_INVALID), (dict(rot=31), B.ERR_INVALID), (dict(rot=0), B.ERR_INVALID),
    (dict(pairs=2), B.ERR_INVALID), (dict(flags=2), B.ERR_INVALID), (dict(n=-1), B.ERR_INVALID),
    (dict(n=11), B.ERR_BOUNDS), (dict(cx=2559), B.ERR_BOUNDS), (dict(cy=2559), B.ERR_BOUNDS),
    (dict(cp=9), B.ERR_BOUNDS), (dict(Lp="(5,2):(1,0)", cp=4), B.ERR_BOUNDS),
    (dict(Lp="(5,3):(1,0)"), B.ERR_SIZE_MISMATCH), (dict(Ly="(64,4,9):(1,64,256)"), B.ERR_SIZE_MISMATCH),
    (dict(Ly="(64,5,10):(1,64,320)", cy=3200), B.ERR_SIZE_MISMATCH),
    (dict(Lx="(64,40):(1,64)"), B.ERR_INVALID), (dict(Lx="Sw<1,3,3> o (64,4,10):(1,64,256)", cx=4096), B.ERR_SWIZZLE),
    (dict(Lx="((8,8),4,10):((1,16),128,512)", cx=9999), B.ERR_INVALID),
    (dict(Ly="(64,4,10):(1,64,0)"), B.ERR_ALIAS), (dict(Ly="(64,4,10):(1,32,256)"), B.ERR_ALIAS),
    (dict(y=X + 64), B.ERR_OVERLAP), (dict(y=X, Ly="(64,4,10):(1,640,64)"), B.ERR_OVERLAP),
    (dict(Lx="(64,4,2147483648):(1,0,0)", Ly="(64,4,2147483648):(1,0,0)"), B.ERR_OVERFLOW)])
def test_rope_refusals(kw, code):
    assert rope(**kw) == code


def test_rope_without_tokens():
    assert rope(n=0) == B.OK and rope(n=0, y=X) == B.OK


def cache(dtype=B.E4M3, **kw):
    a = dict(k=X, v=V, Lk="(64,2,16,8):(1,64,128,2048)", Lv="(64,2,16,8):(1,64,128,2048)", ck=16384, cv=16384,
             ks=W, vs=W + 4096, Ls="(2,16,8):(1,2,32)", cs=256)
    if dtype not in (B.E4M3, B.INT8):
        a.update(ks=None, vs=None)
    a.update(kw)
    c = B.lr_cache()
    c.k, c.v, c.k_scale, c.v_scale, c.dtype = a["k"], a["v"], a["ks"], a["vs"], dtype
    c.k_layout, c.v_layout, c.scale_layout = (lr.Layout(a[n]).c for n in ("Lk", "Lv", "Ls"))
    c.k_capacity, c.v_capacity, c.scale_capacity = a["ck"], a["cv"], a["cs"]
    return c


@pytest.mark.parametrize("kw,code", [
    (dict(), B.OK), (dict(dtype=B.BF16), B.OK), (dict(k=None), B.ERR_INVALID), (dict(v=None), B.ERR_INVALID),
    (dict(ks=None), B.ERR_INVALID), (dict(dtype=B.F16, vs=W), B.ERR_INVALID), (dict(dtype=7), B.ERR_TYPE),
    (dict(ck=16383), B.ERR_BOUNDS), (dict(cs=255), B.ERR_BOUNDS), (dict(Lk="(64,2,16):(1,64,128)"), B.ERR_INVALID),
    (dict(Lv="(64,2,16,7):(1,64,128,2048)"), B.ERR_SIZE_MISMATCH), (dict(Lv="(32,2,16,8):(1,32,64,1024)"), B.OK),
    (dict(Lv="(64,4,8,8):(1,64,256,2048)"), B.ERR_SIZE_MISMATCH), (dict(Ls="(2,16,7):(1,2,32)"), B.ERR_SIZE_MISMATCH),
    (dict(Lk="(64,2,16,8):(1,64,128,0)"), B.ERR_ALIAS), (dict(Ls="(2,16,8):(1,1,32)"), B.ERR_ALIAS),
    (dict(v=X + 8192), B.ERR_OVERLAP), (dict(vs=W + 512), B.ERR_OVERLAP),
    (dict(Lk="(514,2,16,8):(1,514,1028,16448)", ck=999999), B.ERR_INVALID),
    (dict(Lk="Sw<1,3,3> o (64,2,16,8):(1,64,128,2048)"), B.ERR_SWIZZLE)])
def test_cache_checks(kw, code):
    assert lr.lib().lr_cache_validate(cache(**kw)) == code
    assert lr.lib().lr_cache_validate(None) == B.ERR_INVALID


def write(read=False, c=None, **kw):
    a = dict(k=Y, v=Y + 0x100000, Lk="(64,2,10):(1,64,128)", Lv="(64,2,10):(1,64,128)", ck=1280, cv=1280, dtype=B.BF16,
             slots=S, n=10, rot=None)
    a.update(kw)
    c = c if c is not None else cache()
    r = B.lr_rotation(S, S, a["rot"], 0, 1.0) if a["rot"] is not None else None
    Lk, Lv = lr.Layout(a["Lk"]).c, lr.Layout(a["Lv"]).c
    if read:
        return lr.lib().lr_cache_read(c, a["slots"], a["n"], a["k"], Lk, a["ck"], a["v"], Lv, a["cv"], a["dtype"], None)
    return lr.lib().lr_cache_write(c, a["k"], Lk, a["ck"], a["v"], Lv, a["cv"], a["dtype"], a["slots"], a["n"], r, None)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(n=0), B.OK), (dict(n=0, slots=None), B.OK), (dict(n=-1), B.ERR_INVALID), (dict(slots=None), B.ERR_INVALID),
    (dict(k=None), B.ERR_INVALID), (dict(v=None), B.ERR_INVALID), (dict(dtype=B.INT8), B.ERR_TYPE),
    (dict(n=11), B.ERR_BOUNDS), (dict(cv=1279), B.ERR_BOUNDS), (dict(Lk="(32,2,10):(1,64,128)"), B.ERR_SIZE_MISMATCH),
    (dict(Lv="(64,1,10):(1,64,128)"), B.ERR_SIZE_MISMATCH), (dict(Lv="(64,20):(1,64)"), B.ERR_INVALID),
    (dict(k=X + 100), B.ERR_OVERLAP), (dict(v=V), B.ERR_OVERLAP), (dict(v=W + 4100), B.ERR_OVERLAP)])
def test_cache_row_refusals(read, kw, code):
    assert write(read, **kw) == code


def test_cache_pair_refusals():
    assert write(c=cache(B.F16)) == B.ERR_TYPE and write(c=cache(B.F32)) == B.ERR_TYPE
    assert write(rot=66) == B.ERR_INVALID and write(rot=0) == B.ERR_INVALID
    assert write(c=cache(k=None)) == B.ERR_INVALID
    # rows that repeat (a broadcast) may be written from, not read into
    assert write(n=0, Lk="(64,2,10):(1,0,128)") == B.OK
    assert write(read=True, Lk="(64,2,10):(1,0,128)") == B.ERR_ALIAS
    assert write(read=True, v=Y + 64) == B.ERR_OVERLAP


def attend(c=None, plan=False, **kw):
    a = dict(q=Y, Lq="(64,8,3):(1,64,512)", cq=1536, table=S, stride=4, pages=4, lens=S + 4096, batch=3, out=Y + 0x100000,
             Lo="(64,8,3):(1,64,512)", co=1536, lse=None, dtype=B.BF16, scale=0.125, window=0, ws=Y + 0x200000, wb=1 << 24)
    a.update(kw)
    c = c if c is not None else cache()
    Lq, Lo = lr.Layout(a["Lq"]).c, lr.Layout(a["Lo"]).c
    if plan:
        return lr.lib().lr_paged_attention_plan(Lq, c, Lo, a["pages"], a["dtype"], a["window"], B.lr_attention_plan())
    return lr.lib().lr_paged_attention(a["q"], Lq, a["cq"], c, a["table"], a["stride"], a["pages"], a["lens"], a["batch"],
                                       a["out"], Lo, a["co"], a["lse"], a["dtype"], a["scale"], a["window"], a["ws"],
                                       a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), B.OK), (dict(q=None), B.ERR_INVALID), (dict(out=None), B.ERR_INVALID), (dict(table=None), B.ERR_INVALID),
    (dict(lens=None), B.ERR_INVALID), (dict(batch=-1), B.ERR_INVALID), (dict(batch=4), B.ERR_BOUNDS),
    (dict(scale=math.nan), B.ERR_INVALID), (dict(scale=math.inf), B.ERR_INVALID), (dict(window=-1), B.ERR_INVALID),
    (dict(pages=0), B.ERR_INVALID), (dict(pages=1 << 40), B.ERR_OVERFLOW), (dict(stride=-1), B.ERR_INVALID),
    (dict(cq=1535), B.ERR_BOUNDS), (dict(co=1535), B.ERR_BOUNDS), (dict(dtype=B.E4M3), B.ERR_TYPE),
    (dict(Lq="(32,8,3):(1,64,512)"), B.ERR_SIZE_MISMATCH), (dict(Lo="(64,4,3):(1,64,512)"), B.ERR_SIZE_MISMATCH),
    (dict(Lq="(64,7,3):(1,64,512)", Lo="(64,7,3):(1,64,512)"), B.ERR_SIZE_MISMATCH),
    (dict(Lo="(64,8,3):(1,64,0)"), B.ERR_ALIAS), (dict(out=Y), B.ERR_OVERLAP), (dict(out=X), B.ERR_OVERLAP),
    (dict(lse=Y), B.ERR_OVERLAP), (dict(out=S), B.ERR_OVERLAP), (dict(Lq="(64,(2,4),3):(1,(512,64),2048)"), B.ERR_INVALID)])
def test_attention_refusals(kw, code):
    assert attend(**kw) == code


def test_attention_pair_refusals():
    assert attend(c=cache(B.F16)) == B.ERR_TYPE
    big = "(288,2,16,8):(1,288,576,9216)"
    c = cache(B.BF16, Lk=big, Lv=big, ck=73728, cv=73728)
    q = "(288,8,3):(1,288,2304)"
    assert attend(c=c, Lq=q, Lo=q, cq=6912, co=6912) == B.ERR_INVALID    # heads over 256 wide
    assert attend(plan=True, c=c, Lq=q, Lo=q) == B.ERR_INVALID
    assert attend(plan=True) == B.OK and attend(plan=True, window=1 << 62) == B.OK
    assert lr.lib().lr_paged_attention_plan(None, cache(), None, 1, B.BF16, 0, None) == B.ERR_INVALID


def plan_of(c, Lq, max_pages, window=0, dtype=B.BF16):
    p = B.lr_attention_plan()
    assert lr.lib().lr_paged_attention_plan(lr.Layout(Lq).c, c, lr.Layout(Lq).c, max_pages, dtype, window, p) == B.OK
    return p


def test_attention_plan():
    """Chunks cover the longest sequence, the workspace holds every part, and a call without it is refused."""
    rng = random.Random(3)
    for _ in range(300):
        heads, batch, pages = 2 * rng.randint(1, 40), rng.randint(1, 200), rng.randint(1, 20000)
        window = rng.choice([0, 0, 1, 500, 100000])
        p = plan_of(cache(), f"(64,{heads},{batch}):(1,64,{64 * heads})", pages, window)
        span = pages * 16 if not window else min(pages * 16, window + 31)
        assert p.chunk >= 1 and (p.splits - 1) * p.chunk < span <= p.splits * p.chunk
        assert p.workspace_bytes == (0 if p.splits == 1 else batch * heads * p.splits * 66 * 4)
    p = plan_of(cache(), "(64,8,3):(1,64,512)", 4000)
    assert p.splits > 1
    assert attend(pages=4000, stride=4000, wb=p.workspace_bytes - 1, table=0x10000000) == B.ERR_CAPACITY
    assert attend(pages=4000, stride=4000, ws=None, table=0x10000000) == B.ERR_CAPACITY
    assert attend(pages=4000, stride=4000, ws=Y + 0x200004, table=0x10000000) == B.ERR_INVALID
    assert attend(pages=4000, stride=4000, ws=Y, table=0x10000000) == B.ERR_OVERLAP


def test_binding_refusals():
    """What the binding itself refuses: tensors that are not on a GPU, unknown types and names."""
    x = torch.zeros(640)
    t = lr.rope_table(64, device="cpu")
    with pytest.raises(ValueError):
        lr.rope(x, "(64,1,10):(1,64,64)", x, "(64,1,10):(1,64,64)", torch.arange(10), t)
    with pytest.raises(ValueError):
        lr.PagedCache(x, "(64,1,10,1):(1,64,64,640)", x, "(64,1,10,1):(1,64,64,640)")
    with pytest.raises(ValueError):
        B._dtype_code(torch.float64)
    with pytest.raises(ValueError):
        B._rotation(t, torch.arange(3), "thirds")
    with pytest.raises(TypeError):
        B._rotation(t, torch.arange(3, dtype=torch.int32), "half")


def test_structs_match_the_header():
    """The binding's structures have the C sizes (a field added on one side only would shift the rest)."""
    assert ctypes.sizeof(B.lr_rope_params) == 48 and ctypes.sizeof(B.lr_rotation) == 32
    assert ctypes.sizeof(B.lr_attention_plan) == 32
    assert ctypes.sizeof(B.lr_cache) == 4 * 8 + 3 * ctypes.sizeof(B.lr_layout) + 4 * 8


def test_calls_of_nothing():
    """Without a token or a sequence the arrays that have an entry for each may be absent."""
    assert attend(batch=0, lens=None, table=None) == B.OK
    assert attend(batch=0, lens=None) == B.OK and attend(batch=0, table=None) == B.OK
    assert attend(batch=0, lens=None, table=None, q=None) == B.ERR_INVALID
    assert attend(batch=0, lens=None, table=None, pages=0) == B.ERR_INVALID
    assert rope(n=0, positions=None) == B.OK
    assert rope(n=0, positions=None, turns=None) == B.ERR_INVALID and rope(n=0, positions=None, rot=66) == B.ERR_INVALID
    L = lr.Layout("(64,2,10):(1,64,128)").c

    def written(n, positions, turns=S):
        return lr.lib().lr_cache_write(cache(), Y, L, 1280, Y + 0x100000, L, 1280, B.BF16, S if n else None, n,
                                       B.lr_rotation(turns, positions, 64, 0, 1.0), None)
    assert written(0, None) == B.OK and written(0, S) == B.OK
    assert written(10, None) == B.ERR_INVALID and written(0, None, turns=None) == B.ERR_INVALID


@pytest.mark.parametrize("at", [0, -8, 40])
def test_overlap_of_outputs_with_indexes_and_tables(at):
    """Positions, frequencies and slots are inputs too, and a cache's scales are no part of its codes."""
    code = B.ERR_OVERLAP
    assert rope(n=0, positions=Y + at) == code                       # 10 positions
    assert rope(n=0, positions=Y + 5120) == B.OK and rope(n=0, positions=Y - 80) == B.OK
    assert rope(n=0, turns=Y + at) == code                           # 32 frequencies
    assert rope(n=0, turns=Y + 5120) == B.OK and rope(n=0, turns=Y - 256) == B.OK
    assert rope(n=0, positions=Y + at, Lp="(5,2):(1,0)") == code
    assert rope(n=0, x=Y, positions=Y + at) == code                  # in place
    L = lr.Layout("(64,2,10):(1,64,128)").c

    def written(slots=S, positions=S, turns=S, n=10):
        return lr.lib().lr_cache_write(cache(), Y, L, 1280, Y + 0x100000, L, 1280, B.BF16, slots, n,
                                       B.lr_rotation(turns, positions, 64, 0, 1.0), None)
    for first in (X, V, W, W + 4096):                                # codes of keys and values, their scales
        assert written(slots=first + at) == code and written(positions=first + at) == code
        assert written(turns=first + at, n=0) == code
    assert write(read=True, slots=Y + at) == code and write(read=True, slots=Y + 0x100000 + at) == code
    for kw in (dict(ks=X + 16 + at), dict(vs=X + 16 + at), dict(ks=V + 16 + at), dict(vs=V + 16 + at)):
        assert lr.lib().lr_cache_validate(cache(**kw)) == code
    assert lr.lib().lr_cache_validate(cache(ks=X + 16384, vs=V + 16384)) == B.OK
