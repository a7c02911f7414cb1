"""Host side of the operators for long and many-sided contexts (no GPU): the tables of positions with several axes,
the plans, and every refusal.

Refusals are checked before anything is launched, so made-up pointers do: nothing is read through them.
"""

import ctypes
import math

import pytest

import layout_remapping_copy_amd as lr
from layout_remapping_copy_amd import binding as B

torch = pytest.importorskip("torch")


# -------------------------------------------------------------------------------- tables of several axes
def plain_turns(rot, **kw):
    return lr.rope_table(rot, device="cpu", **kw).turns.tolist()


def axis_of(i, sections, order):
    """The axis of pair i, straight from the definition."""
    if order == "blocks":
        return next(a for a in range(len(sections)) if i < sum(sections[:a + 1]))
    a = i % len(sections)
    return a if a and i < len(sections) * sections[a] else 0


@pytest.mark.parametrize("order", ["blocks", "cyclic"])
@pytest.mark.parametrize("sections", [[8], [24, 20, 20], [16, 24, 24], [3, 2, 2], [1, 1], [20, 20], [4, 0, 3], [2, 1, 1, 1],
                                      [256, 128, 128], [0, 5]])
def test_axes_tables(sections, order):
    rot = 2 * sum(sections)
    if order == "cyclic" and any(s and a + (s - 1) * len(sections) >= rot // 2 for a, s in enumerate(sections) if a):
        with pytest.raises(lr.LayoutRemapError):
            lr.rope_axes_table(rot, sections, order=order, device="cpu")
        return
    want = [axis_of(i, sections, order) for i in range(rot // 2)]
    assert [want.count(a) for a in range(len(sections))] == sections
    kw = dict(base=500000.0, scaling="bands", factor=4.0, original_len=8192, low=1.0, high=4.0)
    t = lr.rope_axes_table(rot, sections, order=order, device="cpu", **kw)
    assert t.axis.tolist() == want and t.axes == len(sections) and t.rot_dim == rot and t.magnitude == 1.0
    assert t.turns.tolist() == plain_turns(rot, **kw)
    own = lr.rope_axes_table(rot, sections, order=order, own=True, device="cpu", **kw)
    assert own.axis.tolist() == want
    for a, s in enumerate(sections):
        mine = [own.turns.tolist()[i] for i in range(rot // 2) if want[i] == a]
        assert mine == (plain_turns(2 * s, **kw) if s else [])


def test_axes_magnitude():
    t = lr.rope_axes_table(64, [16, 16], scaling="parts", factor=8.0, original_len=4096, device="cpu")
    assert abs(t.magnitude - (0.1 * math.log(8.0) + 1)) < 1e-15


@pytest.mark.parametrize("kw", [dict(sections=[]), dict(sections=[32, 1]), dict(sections=[31]), dict(sections=[33, -1]),
                                dict(sections=[8, 8, 8, 4, 4]), dict(rot=0, sections=[0]), dict(rot=63), dict(rot=1026),
                                dict(sections=[8, 24], order="cyclic"), dict(base=1.0),
                                dict(scaling="linear", factor=0.0), dict(scaling="linear", factor=0.0, own=True)])
def test_axes_table_refusals(kw):
    kw = dict(kw)
    with pytest.raises(lr.LayoutRemapError) as e:
        lr.rope_axes_table(kw.pop("rot", 64), kw.pop("sections", [16, 16]), device="cpu", **kw)
    assert e.value.code == B.ERR_INVALID


def test_axes_table_arguments():
    p, s = B.lr_rope_params(4, 0, 10000.0, 1.0, 0.0, 1.0, 32.0), (ctypes.c_int32 * 2)(1, 1)
    turns, axis, m = (ctypes.c_int64 * 2)(), (ctypes.c_int32 * 2)(), ctypes.c_double()

    def call(p=p, s=s, axes=2, order=0, spectrum=0, turns=turns, axis=axis, m=m):
        return lr.lib().lr_rope_axes_table(p, s, axes, order, spectrum, turns, axis, m)
    assert call() == B.OK
    for kw in (dict(p=None), dict(s=None), dict(turns=None), dict(axis=None), dict(m=None), dict(axes=0), dict(axes=5),
               dict(axes=-1), dict(order=2), dict(order=-1), dict(spectrum=2), dict(spectrum=-1)):
        assert call(**kw) == B.ERR_INVALID
    with pytest.raises(ValueError):
        lr.rope_axes_table(64, [32], order="rows", device="cpu")
    with pytest.raises(ValueError):
        lr.rope_axes_table(64, [32], scaling="twice", device="cpu")


# -------------------------------------------------------------------------------- refusals: several axes
X, Y, V, W, S = 0x100000, 0x40000000, 0x80000000, 0xc0000000, 0x200000  # far apart, never read
A = S + 0x10000


def rope_axes(**kw):
    a = dict(x=X, Lx="(64,4,10):(1,64,256)", cx=2560, y=Y, Ly="(64,4,10):(1,64,256)", cy=2560, dtype=B.BF16,
             turns=S, axis=A, positions=S + 0x1000, rot=64, pairs=0, axes=3, Lp=None, cp=30, n=10, flags=0)
    a.update(kw)
    lay = {k: (lr.Layout(a[k]).c if a[k] is not None else None) for k in ("Lx", "Ly", "Lp")}
    r = B.lr_axes_rotation(a["turns"], a["axis"], a["positions"], a["rot"], a["pairs"], a["axes"], 1.0) if a["rot"] is not None else None
    return lr.lib().lr_rope_axes(a["x"], lay["Lx"], a["cx"], a["y"], lay["Ly"], a["cy"], a["dtype"], r, lay["Lp"], a["cp"],
                                 a["n"], a["flags"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), B.ERR_INVALID), (dict(y=None), B.ERR_INVALID), (dict(Lx=None), B.ERR_INVALID),
    (dict(rot=None), B.ERR_INVALID), (dict(turns=None), B.ERR_INVALID), (dict(positions=None), B.ERR_INVALID),
    (dict(axis=None), B.ERR_INVALID), (dict(axes=0), B.ERR_INVALID), (dict(axes=5), B.ERR_INVALID),
    (dict(dtype=B.INT8), B.ERR_TYPE), (dict(rot=66), B.ERR_INVALID), (dict(rot=31), B.ERR_INVALID),
    (dict(pairs=-1), B.ERR_INVALID), (dict(flags=4), B.ERR_INVALID), (dict(n=-1), B.ERR_INVALID),
    (dict(n=11, cp=33), B.ERR_BOUNDS), (dict(cp=29), B.ERR_BOUNDS), (dict(cx=2559), B.ERR_BOUNDS),
    (dict(Lp="(10,3):(1,10)", n=0), B.OK), (dict(Lp="(10,3):(1,10)", cp=29), B.ERR_BOUNDS),
    (dict(Lp="(10,2):(1,10)"), B.ERR_SIZE_MISMATCH), (dict(Lp="(9,3):(1,10)"), B.ERR_SIZE_MISMATCH),
    (dict(Lp="10:1"), B.ERR_INVALID), (dict(Lp="(10,3,1):(1,10,0)"), B.ERR_INVALID),
    (dict(Lp="(10,(2,2)):(1,(10,30))", axes=4, cp=99), B.ERR_INVALID),
    (dict(Ly="(64,4,9):(1,64,256)"), B.ERR_SIZE_MISMATCH), (dict(Ly="(64,4,10):(1,64,0)"), B.ERR_ALIAS),
    (dict(y=X + 64), B.ERR_OVERLAP)])
def test_rope_axes_refusals(kw, code):
    assert rope_axes(**kw) == code


@pytest.mark.parametrize("at", [0, -8, 40])
def test_rope_axes_overlap(at):
    assert rope_axes(n=0, positions=Y + at) == B.ERR_OVERLAP and rope_axes(n=0, positions=Y - 240) == B.OK
    assert rope_axes(n=0, axis=Y + at) == B.ERR_OVERLAP and rope_axes(n=0, axis=Y - 128) == B.OK
    assert rope_axes(n=0, turns=Y + at) == B.ERR_OVERLAP and rope_axes(n=0, turns=Y - 256) == B.OK
    assert rope_axes(n=0, positions=None, cp=0) == B.OK and rope_axes(n=0, axis=None) == B.ERR_INVALID


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


def write_axes(c=None, **kw):
    a = dict(k=Y, v=Y + 0x100000, L="(64,2,10):(1,64,128)", dtype=B.BF16, slots=S, n=10, turns=S + 0x1000, axis=A,
             positions=S + 0x2000, rot=64, pairs=0, axes=2)
    a.update(kw)
    c = c if c is not None else cache()
    r = B.lr_axes_rotation(a["turns"], a["axis"], a["positions"], a["rot"], a["pairs"], a["axes"], 1.0) if a["rot"] is not None else None
    L = lr.Layout(a["L"]).c
    return lr.lib().lr_cache_write_axes(c, a["k"], L, 1280, a["v"], L, 1280, a["dtype"], a["slots"], a["n"], r, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), B.OK), (dict(rot=None), B.ERR_INVALID), (dict(axes=0), B.ERR_INVALID), (dict(axes=5), B.ERR_INVALID),
    (dict(axis=None), B.ERR_INVALID), (dict(turns=None), B.ERR_INVALID), (dict(positions=None), B.ERR_INVALID),
    (dict(rot=66), B.ERR_INVALID), (dict(n=-1), B.ERR_INVALID), (dict(n=11), B.ERR_BOUNDS), (dict(dtype=B.E4M3), B.ERR_TYPE),
    (dict(axis=X), B.ERR_OVERLAP), (dict(axis=W - 64, n=0), B.ERR_OVERLAP), (dict(positions=V - 80), B.ERR_OVERLAP),
    (dict(positions=V - 160, n=0), B.OK), (dict(turns=W + 4096), B.ERR_OVERLAP), (dict(slots=X), B.ERR_OVERLAP)])
def test_write_axes_refusals(kw, code):
    assert write_axes(**kw) == code


def test_axes_binding_refusals():
    x, t = torch.zeros(640), lr.rope_axes_table(64, [16, 16], device="cpu")
    with pytest.raises(ValueError):
        lr.rope_axes(x, "(64,1,10):(1,64,64)", x, "(64,1,10):(1,64,64)", torch.zeros(2, 10, dtype=torch.int64), t)
    with pytest.raises(ValueError):
        B._axes_rotation(t, torch.arange(3), "thirds")
    with pytest.raises(TypeError):
        B._axes_rotation(t, torch.arange(3, dtype=torch.int32), "half")
    assert ctypes.sizeof(B.lr_axes_rotation) == 40


# -------------------------------------------------------------------------------- refusals: a shared prefix
def prefix(c=None, plan=False, **kw):
    a = dict(q=Y, Lq="(64,8,3):(1,64,512)", cq=1536, prefix=A, pp=4, plen=A + 0x1000, table=S, stride=4, pages=4, lens=S + 4096,
             batch=3, out=Y + 0x100000, Lo="(64,8,3):(1,64,512)", co=1536, lse=None, dtype=B.BF16, scale=0.125, ws=Y + 0x200000,
             wb=1 << 24)
    a.update(kw)
    c = c if c is not None else cache()
    Lq, Lo = lr.Layout(a["Lq"]).c, lr.Layout(a["Lo"]).c
    if plan:
        return lr.lib().lr_prefix_attention_plan(Lq, c, Lo, a["pp"], a["pages"], a["dtype"], B.lr_prefix_plan())
    return lr.lib().lr_prefix_attention(a["q"], Lq, a["cq"], c, a["prefix"], a["pp"], a["plen"], a["table"], a["stride"],
                                        a["pages"], a["lens"], a["batch"], a["out"], Lo, a["co"], a["lse"], a["dtype"],
                                        a["scale"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), B.OK), (dict(batch=0, prefix=None, plen=None, table=None, lens=None), B.OK),
    (dict(q=None), B.ERR_INVALID), (dict(out=None), B.ERR_INVALID), (dict(table=None), B.ERR_INVALID),
    (dict(lens=None), B.ERR_INVALID), (dict(prefix=None), B.ERR_INVALID), (dict(plen=None), B.ERR_INVALID),
    (dict(batch=-1), B.ERR_INVALID), (dict(batch=4), B.ERR_BOUNDS), (dict(scale=math.nan), B.ERR_INVALID),
    (dict(scale=math.inf), B.ERR_INVALID), (dict(pages=0), B.ERR_INVALID), (dict(pp=0), B.ERR_INVALID),
    (dict(pp=-1), B.ERR_INVALID), (dict(pages=1 << 40), B.ERR_OVERFLOW), (dict(pp=1 << 40), B.ERR_OVERFLOW),
    (dict(stride=-1), B.ERR_INVALID), (dict(cq=1535), B.ERR_BOUNDS), (dict(co=1535), B.ERR_BOUNDS),
    (dict(dtype=B.E4M3), B.ERR_TYPE), (dict(Lq="(32,8,3):(1,64,512)"), B.ERR_SIZE_MISMATCH),
    (dict(Lo="(64,4,3):(1,64,512)"), B.ERR_SIZE_MISMATCH),
    (dict(Lq="(64,7,3):(1,64,512)", Lo="(64,7,3):(1,64,512)"), B.ERR_SIZE_MISMATCH),
    (dict(Lo="(64,8,3):(1,64,0)"), B.ERR_ALIAS), (dict(out=Y), B.ERR_OVERLAP), (dict(out=X), B.ERR_OVERLAP),
    (dict(lse=Y), B.ERR_OVERLAP), (dict(out=S), B.ERR_OVERLAP), (dict(out=A - 8), B.ERR_OVERLAP), (dict(lse=A + 0x1000), B.ERR_OVERLAP),
    (dict(lse=A - 92), B.ERR_OVERLAP), (dict(ws=Y, batch=0), B.ERR_OVERLAP), (dict(ws=A & ~15), B.ERR_OVERLAP),
    (dict(ws=None), B.ERR_CAPACITY), (dict(wb=100), B.ERR_CAPACITY), (dict(ws=Y + 0x200004), B.ERR_INVALID),
    (dict(Lq="(64,(2,4),3):(1,(512,64),2048)", cq=9999), B.ERR_INVALID)])
def test_prefix_refusals(kw, code):
    assert prefix(**kw) == code


def test_prefix_pairs_and_plan():
    assert prefix(c=cache(B.F16)) == B.ERR_TYPE
    big = "(288,2,16,8):(1,288,576,9216)"
    c = cache(B.BF16, Lk=big, Lv=big, ck=73728, cv=73728)
    q = "(288,8,3):(1,288,2304)"
    assert prefix(c=c, Lq=q, Lo=q, cq=6912, co=6912) == B.ERR_INVALID and prefix(plan=True, c=c, Lq=q, Lo=q) == B.ERR_INVALID
    assert prefix(plan=True) == B.OK
    assert lr.lib().lr_prefix_attention_plan(None, cache(), None, 1, 1, B.BF16, None) == B.ERR_INVALID
    for heads, batch, pp, pages in ((8, 3, 1, 1), (8, 1, 4000, 1), (64, 128, 2048, 128), (2, 200, 20000, 3), (80, 7, 3, 5000)):
        p = B.lr_prefix_plan()
        L = lr.Layout(f"(64,{heads},{batch}):(1,64,{64 * heads})").c
        assert lr.lib().lr_prefix_attention_plan(L, cache(), L, pp, pages, B.BF16, p) == B.OK
        parts = batch * heads * (p.prefix_splits + p.own_splits)
        assert p.prefix_splits >= 1 and p.own_splits >= 1
        assert parts * 66 * 4 <= p.workspace_bytes <= parts * 66 * 4 + 64
        n = 64 * heads * batch
        args = dict(Lq=f"(64,{heads},{batch}):(1,64,{64 * heads})", Lo=f"(64,{heads},{batch}):(1,64,{64 * heads})", cq=n, co=n,
                    pp=pp, pages=pages, stride=pages, batch=0, out=Y + (1 << 28), ws=Y + (1 << 29))
        assert prefix(wb=p.workspace_bytes, **args) == B.OK and prefix(wb=p.workspace_bytes - 1, **args) == B.ERR_CAPACITY


# -------------------------------------------------------------------------------- refusals: blocks
def keys(c=None, **kw):
    a = dict(slots=S, n=10, keys=Y, L="(64,2,8):(1,64,128)", cap=1024, dtype=B.BF16)
    a.update(kw)
    c = c if c is not None else cache()
    return lr.lib().lr_block_keys(c, a["slots"], a["n"], a["keys"], lr.Layout(a["L"]).c if a["L"] else None, a["cap"], a["dtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), B.OK), (dict(n=0, slots=None), B.OK), (dict(n=-1), B.ERR_INVALID), (dict(slots=None), B.ERR_INVALID),
    (dict(keys=None), B.ERR_INVALID), (dict(L=None), B.ERR_INVALID), (dict(dtype=B.INT8), B.ERR_TYPE), (dict(cap=1023), B.ERR_BOUNDS),
    (dict(L="(32,2,8):(1,64,128)"), B.ERR_SIZE_MISMATCH), (dict(L="(64,1,8):(1,64,128)"), B.ERR_SIZE_MISMATCH),
    (dict(L="(64,2,7):(1,64,128)"), B.ERR_SIZE_MISMATCH), (dict(L="(64,16):(1,64)"), B.ERR_INVALID),
    (dict(L="(64,2,8):(1,64,0)"), B.ERR_ALIAS), (dict(L="(64,2,8):(1,32,128)"), B.ERR_ALIAS),
    (dict(L="((8,8),2,8):((1,16),256,512)", cap=9999), B.ERR_INVALID), (dict(keys=S), B.ERR_OVERLAP), (dict(keys=X + 64), B.ERR_OVERLAP),
    (dict(keys=V), B.ERR_OVERLAP), (dict(keys=W + 4096), B.ERR_OVERLAP), (dict(n=1 << 31), B.ERR_OVERFLOW)])
def test_block_keys_refusals(kw, code):
    assert keys(**kw) == code


def test_block_keys_pairs():
    assert keys(c=cache(B.F16), n=0) == B.ERR_TYPE and keys(c=cache(B.BF16), n=0) == B.OK
    assert keys(c=cache(k=None)) == B.ERR_INVALID and keys(dtype=B.F32, n=0) == B.OK
    assert keys(n=0, L="(64,2,8):(16,1024,2)", cap=4096) == B.OK        # any order of the head dimension, heads and pages


def select(plan=False, **kw):
    a = dict(q=Y, Lq="(64,8,3):(1,64,512)", cq=1536, keys=V, Lk="(64,2,9):(1,64,128)", ck=1152, dtype=B.BF16, table=S, stride=40,
             pages=40, lens=S + 4096, page=16, batch=3, first=1, last=2, blocks=W, count=8, ws=Y + 0x200000, wb=3 * 2 * 40 * 8)
    a.update(kw)
    Lq, Lk = lr.Layout(a["Lq"]).c, lr.Layout(a["Lk"]).c
    if plan:
        n = ctypes.c_int64()
        return lr.lib().lr_block_select_plan(Lq, Lk, a["pages"], n), n.value
    return lr.lib().lr_block_select(a["q"], Lq, a["cq"], a["keys"], Lk, a["ck"], a["dtype"], a["table"], a["stride"], a["pages"],
                                    a["lens"], a["page"], a["batch"], a["first"], a["last"], a["blocks"], a["count"], a["ws"],
                                    a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), B.OK), (dict(batch=0, table=None, lens=None), B.OK), (dict(q=None), B.ERR_INVALID), (dict(keys=None), B.ERR_INVALID),
    (dict(blocks=None), B.ERR_INVALID), (dict(table=None), B.ERR_INVALID), (dict(lens=None), B.ERR_INVALID),
    (dict(batch=-1), B.ERR_INVALID), (dict(batch=4), B.ERR_BOUNDS), (dict(stride=-1), B.ERR_INVALID), (dict(pages=0), B.ERR_INVALID),
    (dict(page=0), B.ERR_INVALID), (dict(page=-1), B.ERR_INVALID), (dict(page=1 << 31), B.ERR_OVERFLOW), (dict(count=0), B.ERR_INVALID),
    (dict(first=-1), B.ERR_INVALID), (dict(last=-1), B.ERR_INVALID), (dict(first=7), B.ERR_INVALID), (dict(first=9, last=0), B.ERR_INVALID),
    (dict(first=(1 << 63) - 1, last=(1 << 63) - 1), B.ERR_INVALID), (dict(first=6, batch=0), B.OK), (dict(count=1 << 31, batch=0), B.ERR_OVERFLOW),
    (dict(dtype=B.E4M3), B.ERR_TYPE), (dict(cq=1535), B.ERR_BOUNDS), (dict(ck=1151), B.ERR_BOUNDS),
    (dict(Lk="(32,2,9):(1,64,128)"), B.ERR_SIZE_MISMATCH), (dict(Lk="(64,3,9):(1,64,128)"), B.ERR_BOUNDS),
    (dict(Lk="(64,3,9):(1,64,192)", ck=1728), B.ERR_SIZE_MISMATCH),
    (dict(Lk="(64,18):(1,64)"), B.ERR_INVALID), (dict(Lq="(288,8,3):(1,288,2304)", Lk="(288,2,9):(1,288,576)", cq=9999, ck=9999), B.ERR_INVALID),
    (dict(ws=None), B.ERR_CAPACITY), (dict(wb=1919), B.ERR_CAPACITY), (dict(ws=Y + 0x200008), B.ERR_INVALID),
    (dict(blocks=Y), B.ERR_OVERLAP), (dict(blocks=V + 2300), B.ERR_OVERLAP), (dict(blocks=S + 4), B.ERR_OVERLAP),
    (dict(blocks=S + 4096), B.ERR_OVERLAP), (dict(ws=W), B.ERR_OVERLAP), (dict(ws=V), B.ERR_OVERLAP),
    (dict(Lk="(64,2,9):(1,64,0)", batch=0), B.OK)])
def test_block_select_refusals(kw, code):
    assert select(**kw) == code


def test_block_select_plan():
    assert select(plan=True) == (B.OK, 3 * 2 * 40 * 8) and select(plan=True, pages=1) == (B.OK, 48)
    assert select(plan=True, pages=0)[0] == B.ERR_INVALID and select(plan=True, pages=1 << 31)[0] == B.ERR_OVERFLOW
    L = lr.Layout("(64,8,3):(1,64,512)").c
    assert lr.lib().lr_block_select_plan(L, L, 4, None) == B.ERR_INVALID


def attend_blocks(c=None, plan=False, **kw):
    a = dict(q=Y, Lq="(64,8,3):(1,64,512)", cq=1536, blocks=A, count=5, table=S, stride=40, pages=40, lens=S + 4096, batch=3,
             out=Y + 0x100000, Lo="(64,8,3):(1,64,512)", co=1536, lse=None, dtype=B.BF16, scale=0.125, ws=Y + 0x200000, wb=1 << 24)
    a.update(kw)
    c = c if c is not None else cache()
    Lq, Lo = lr.Layout(a["Lq"]).c, lr.Layout(a["Lo"]).c
    if plan:
        p = B.lr_attention_plan()
        return lr.lib().lr_block_attention_plan(Lq, c, Lo, a["count"], a["dtype"], p), p
    return lr.lib().lr_block_attention(a["q"], Lq, a["cq"], c, a["blocks"], a["count"], a["table"], a["stride"], a["pages"],
                                       a["lens"], a["batch"], a["out"], Lo, a["co"], a["lse"], a["dtype"], a["scale"], a["ws"],
                                       a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), B.OK), (dict(batch=0, blocks=None, table=None, lens=None), B.OK), (dict(q=None), B.ERR_INVALID),
    (dict(out=None), B.ERR_INVALID), (dict(blocks=None), B.ERR_INVALID), (dict(table=None), B.ERR_INVALID),
    (dict(lens=None), B.ERR_INVALID), (dict(batch=-1), B.ERR_INVALID), (dict(batch=4), B.ERR_BOUNDS),
    (dict(scale=math.inf), B.ERR_INVALID), (dict(pages=0), B.ERR_INVALID), (dict(count=0), B.ERR_INVALID),
    (dict(count=-1), B.ERR_INVALID), (dict(pages=1 << 40), B.ERR_OVERFLOW), (dict(count=1 << 40), B.ERR_OVERFLOW),
    (dict(stride=-1), B.ERR_INVALID), (dict(cq=1535), B.ERR_BOUNDS), (dict(co=1535), B.ERR_BOUNDS), (dict(dtype=B.INT8), B.ERR_TYPE),
    (dict(Lq="(32,8,3):(1,64,512)"), B.ERR_SIZE_MISMATCH), (dict(Lo="(64,8,3):(1,64,0)"), B.ERR_ALIAS), (dict(out=Y), B.ERR_OVERLAP),
    (dict(out=A + 64), B.ERR_OVERLAP), (dict(out=S + 64), B.ERR_OVERLAP), (dict(lse=A - 92), B.ERR_OVERLAP), (dict(out=V), B.ERR_OVERLAP)])
def test_block_attention_refusals(kw, code):
    assert attend_blocks(**kw) == code


def test_block_attention_plan():
    rc, p = attend_blocks(plan=True, count=4000)
    assert rc == B.OK and p.splits > 1 and p.workspace_bytes == 3 * 8 * p.splits * 66 * 4
    assert attend_blocks(count=4000, wb=p.workspace_bytes - 1) == B.ERR_CAPACITY
    assert attend_blocks(count=4000, ws=None) == B.ERR_CAPACITY and attend_blocks(count=4000, ws=Y + 0x200004) == B.ERR_INVALID
    rc, p = attend_blocks(plan=True, count=4)
    assert rc == B.OK and p.splits == 1 and p.workspace_bytes == 0
    assert attend_blocks(c=cache(B.F16)) == B.ERR_TYPE
    assert lr.lib().lr_block_attention_plan(None, cache(), None, 1, B.BF16, None) == B.ERR_INVALID


def test_structs_match_the_header():
    assert ctypes.sizeof(B.lr_prefix_plan) == 32


@pytest.mark.parametrize("heads,batch,pages,tiles", [
    (8, 3, 1, 1), (8, 40, 10, 10), (80, 7, 3, 18),  # 12, 160 and 280 rows of a cache head: tiles of 16
    (8, 40, 1000, 2), (8, 32, 8000, 1),             # 160 and 128 on 16000 and 128000 tokens: of 128
    (64, 16, 300, 2), (64, 9, 2000, 3), (64, 128, 2048, 16)])  # 512 and 4096: of 256; 288 over codes: of 128
def test_prefix_plan_tiles(heads, batch, pages, tiles):
    """The plan says how many workgroups share the prefix's keys as the call will run, not as that of one sequence would."""
    p = B.lr_prefix_plan()
    L = lr.Layout(f"(64,{heads},{batch}):(1,64,{64 * heads})").c
    assert lr.lib().lr_prefix_attention_plan(L, cache(), L, pages, 3, B.BF16, p) == B.OK
    assert p.row_tiles == tiles


def test_blocks_of_no_sequence():
    assert select(batch=0, blocks=None, table=None, lens=None) == B.OK
    assert select(batch=1, blocks=None) == B.ERR_INVALID
    # as many entries as no memory holds, counted without a wrap
    many = "(64,2,1000000000):(1,64,128)"
    assert select(Lq=many, cq=1 << 62, batch=1000000000, count=(1 << 31) - 1, pages=1, ws=Y, wb=1 << 62) == B.ERR_OVERFLOW
