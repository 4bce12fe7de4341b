"""Host side of the position, cache and tree-attention entry points: refusals
before anything is enqueued, frequencies, mask words (no GPU)."""
import ctypes
import math

import pytest
import torch

import exact_attention_14_gb300 as ea


@pytest.fixture(scope="module")
def lib():
    from exact_attention_14_gb300 import _build
    _build.build()
    return ea.load()


FAKE = 0x10000   # aligned, never read: every case is refused first


def strides(*s):
    return (ctypes.c_longlong * 3)(*s)


def rope(lib, **kw):
    a = dict(q=FAKE, k=FAKE, qo=2 * FAKE, ko=2 * FAKE, qs=strides(4096, 1024, 128), ks=strides(2048, 1024, 128),
             qos=strides(4096, 1024, 128), kos=strides(2048, 1024, 128), pos=FAKE, ps=8, f=FAKE, B=2, Hq=4, Hkv=2,
             N=8, d=128, rot=128, inter=0, inv=0, mag=1.0, idt=0, odt=0)
    a.update(kw)
    return lib.attn_rope(a["q"], a["k"], a["qo"], a["ko"], a["qs"], a["ks"], a["qos"], a["kos"], a["pos"], a["ps"],
                         a["f"], a["B"], a["Hq"], a["Hkv"], a["N"], a["d"], a["rot"], a["inter"], a["inv"],
                         a["mag"], a["idt"], a["odt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(qo=None), 1), (dict(pos=None), 1), (dict(f=None), 1), (dict(f=FAKE + 4), 1),
    (dict(q=FAKE + 8), 1), (dict(k=None), 1), (dict(ko=None), 1), (dict(k=None, ko=None), 1), (dict(B=0), 1),
    (dict(N=0), 1), (dict(rot=0), 1), (dict(rot=3), 1), (dict(rot=130), 1), (dict(inter=2), 1), (dict(inv=-1), 1),
    (dict(mag=float("nan")), 1), (dict(ps=-1), 1), (dict(idt=5), 1), (dict(odt=2), 1), (dict(qs=None, d=100, rot=100), 2),
    (dict(qs=strides(4096, 1024, 100)), 1), (dict(qos=strides(4096, 1024, 0)), 1),
    (dict(qos=strides(4096, 1024, 64)), 1), (dict(qos=strides(4096, 64, 128)), 1),
    (dict(qos=strides(2048, 1024, 128)), 1), (dict(qo=FAKE, odt=1), 1),
    (dict(qo=FAKE, qs=strides(4096, 128, 512)), 1), (dict(N=1 << 30), 1),
    (dict(d=12, rot=4), 2), (dict(d=264, rot=4), 2),
])
def test_rope_refusals(lib, kw, code):
    assert rope(lib, **kw) == code


def write(lib, **kw):
    a = dict(k=FAKE, v=FAKE, ks=strides(2048, 1024, 128), vs=strides(2048, 128, 256), kp=FAKE, vp=FAKE, kd=FAKE,
             vd=FAKE, slots=FAKE, B=2, N=8, H=2, d=128, nb=4, page=16, kind=1)
    a.update(kw)
    return lib.attn_cache_write(a["k"], a["v"], a["ks"], a["vs"], a["kp"], a["vp"], a["kd"], a["vd"], a["slots"],
                                a["B"], a["N"], a["H"], a["d"], a["nb"], a["page"], a["kind"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=FAKE + 2), 1), (dict(slots=None), 1), (dict(slots=FAKE + 4), 1), (dict(kp=None), 1),
    (dict(kd=None), 1), (dict(vd=FAKE + 4), 1), (dict(B=0), 1), (dict(N=1 << 30), 1), (dict(H=0), 1),
    (dict(nb=0), 1), (dict(page=0), 1), (dict(kind=2), 1), (dict(ks=strides(2048, 1024, 4)), 1),
    (dict(vs=strides(2048, -128, 256)), 1), (dict(d=72), 2), (dict(d=272), 2), (dict(kind=0, d=100), 2),
])
def test_cache_write_refusals(lib, kw, code):
    assert write(lib, **kw) == code


def read(lib, **kw):
    a = dict(kp=FAKE, vp=FAKE, kd=FAKE, vd=FAKE, table=FAKE, cu=FAKE, ko=FAKE, vo=FAKE, B=2, H=2, total=9, nb=4,
             page=16, mb=2, d=128, kind=1, odt=0)
    a.update(kw)
    return lib.attn_cache_read(a["kp"], a["vp"], a["kd"], a["vd"], a["table"], a["cu"], a["ko"], a["vo"], a["B"],
                               a["H"], a["total"], a["nb"], a["page"], a["mb"], a["d"], a["kind"], a["odt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(kp=None), 1), (dict(table=None), 1), (dict(cu=FAKE + 2), 1), (dict(ko=FAKE + 4), 1), (dict(vo=None), 1),
    (dict(vd=None), 1), (dict(B=0), 1), (dict(total=0), 1), (dict(mb=0), 1), (dict(odt=9), 1), (dict(kind=-1), 1),
    (dict(d=24), 2), (dict(kind=0, d=4), 2), (dict(H=1 << 20), 2),
])
def test_cache_read_refusals(lib, kw, code):
    assert read(lib, **kw) == code


def tree(lib, **kw):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, kd=FAKE, vd=FAKE, table=FAKE, sl=FAKE, ql=None, mask=None, o=FAKE, lse=None,
             B=2, Hq=8, Hkv=2, T=4, nb=4, page=16, mb=2, d=128, scale=0.1, kind=1, ws=FAKE, wsb=1 << 40, odt=1)
    a.update(kw)
    return lib.attn_decode_tree(a["q"], a["kp"], a["vp"], a["kd"], a["vd"], a["table"], a["sl"], a["ql"], a["mask"],
                                a["o"], a["lse"], a["B"], a["Hq"], a["Hkv"], a["T"], a["nb"], a["page"], a["mb"],
                                a["d"], a["scale"], a["kind"], a["ws"], a["wsb"], a["odt"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(q=FAKE + 4), 1), (dict(table=None), 1), (dict(sl=FAKE + 2), 1), (dict(ql=FAKE + 2), 1),
    (dict(mask=FAKE + 4), 1), (dict(lse=FAKE + 2), 1), (dict(o=None), 1), (dict(kd=None), 1), (dict(B=0), 1),
    (dict(Hq=7), 1), (dict(T=0), 1), (dict(mb=0), 1), (dict(mb=1 << 21), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("inf")), 1), (dict(odt=3), 1), (dict(kind=3), 1), (dict(nb=0), 1),
    (dict(T=1025), 2), (dict(page=24), 2), (dict(d=72), 2), (dict(kind=0, d=260), 2),
    (dict(T=1024, Hq=1 << 21, Hkv=1), 2), (dict(T=1024, B=2048, Hq=1024, Hkv=1024), 2),
])
def test_decode_tree_refusals(lib, kw, code):
    assert tree(lib, **kw) == code


def test_tree_workspace_size_refuses(lib):
    for a in [(0, 8, 2, 4, 2, 16, 128), (1, 7, 2, 4, 2, 16, 128), (1, 8, 2, 0, 2, 16, 128), (1, 8, 2, 4, 2, 8, 128),
              (1, 8, 2, 4, 2, 16, 100)]:
        assert ea.attn_decode_tree_workspace_size(*a) == 0
    assert ea.attn_decode_tree_workspace_size(1, 8, 2, 4, 2, 16, 72, True) == 0


def test_binding_refuses_cpu_and_wrong_types(lib):
    x, i = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 4, dtype=torch.int32)
    f = torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError):
        ea.rope(x, None, i, f)                                  # CPU tensors
    with pytest.raises(TypeError):
        ea.rope(x.half(), None, i, f)
    pages = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ea.attn_cache_write(x, x, pages, pages, i.long())
    with pytest.raises(TypeError):
        ea.attn_cache_write(x.float(), x, pages, pages, i.long())
    with pytest.raises(ValueError):
        ea.cache_read(pages, pages, i, i[0], 4)
    with pytest.raises(ValueError):
        ea.decode_tree(x, pages, pages, i, i[0])
    with pytest.raises(ValueError):
        ea.tree_mask_words(torch.zeros(1, 3, 4, dtype=torch.bool))


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (250, 1e6)])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("by_parts", 16.0)])
def test_frequencies(lib, rot, base, scaling, factor):
    got, mag = ea.attn_rope_frequencies(rot, base, scaling=scaling, factor=factor, original_len=4096)
    b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" and rot > 2 else base
    want = [b ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        want = [x / factor for x in want]
    if scaling == "by_parts":
        def at(turns):
            return rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot // 2 - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(rot // 2)]
        want = [x / factor * r + x * (1 - r) for x, r in zip(want, ramp)]
        # the ends: fast pairs kept, slow pairs divided
        assert got[0] == 1.0 or rot == 2
        assert rot < 64 or math.isclose(got[-1], base ** (-2 * (rot // 2 - 1) / rot) / factor, rel_tol=1e-12)
    assert all(math.isclose(x, y, rel_tol=1e-13) for x, y in zip(got, want)) and len(got) == rot // 2
    assert math.isclose(mag, 0.1 * math.log(factor) + 1 if scaling == "by_parts" else 1.0, rel_tol=2.0 ** -23)


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=258), dict(base=1.0),
                                dict(base=float("nan")), dict(scaling="linear", factor=0.5),
                                dict(scaling="by_parts", factor=2.0), dict(scaling="by_parts", factor=2.0,
                                                                           original_len=64, beta_fast=0.5)])
def test_frequencies_refuse(lib, kw):
    a = dict(rotary_dim=64, base=10000.0)
    a.update(kw)
    with pytest.raises(ea.AttnError):
        ea.attn_rope_frequencies(a.pop("rotary_dim"), a.pop("base"), **a)


def test_mask_words(lib):
    m = torch.rand(2, 130, 130, generator=torch.Generator().manual_seed(0)) < 0.5
    w = ea.tree_mask_words(m)
    assert w.shape == (2, 130, 3) and w.dtype == torch.int64
    for b, t, u in [(0, 0, 0), (1, 129, 63), (0, 64, 64), (1, 5, 127), (0, 77, 128), (1, 100, 129)]:
        assert ((int(w[b, t, u // 64]) >> (u % 64)) & 1) == int(m[b, t, u])
