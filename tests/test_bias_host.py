"""Host side of the entry points with a relative position bias and of the paged
cache's tables: refusals before anything is enqueued, the map of distances to
buckets (no GPU)."""
import ctypes
import math

import pytest
import torch

import exact_attention_14_gb300 as ea
from bias_ref import Pages, Problem, bucket


@pytest.fixture(scope="module")
def lib():
    from exact_attention_14_gb300 import _build
    _build.build()
    return ea.load()


FAKE = 0x10000   # aligned, never read: every case is refused first
BIAS = dict(table=FAKE, tt=1, buckets=FAKE, first=-113, span=114, nb=32)
BAD_BIAS = [(dict(table=None), 1), (dict(buckets=None), 1), (dict(table=FAKE + 2), 1), (dict(table=FAKE + 1, tt=0), 1),
            (dict(buckets=FAKE + 2), 1), (dict(tt=2), 1), (dict(span=0), 1), (dict(nb=0), 1),
            (dict(first=-(1 << 24) - 1), 1), (dict(first=(1 << 24) + 1), 1), (dict(span=65537), 2),
            (dict(nb=65537), 2), (dict(d=136), 2), (dict(d=256), 2), (dict(d=12), 2)]


def _bias(a):
    return a["table"], a["tt"], a["buckets"], a["first"], a["span"], a["nb"]


def fwd(lib, **kw):
    a = dict(BIAS, q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, B=1, Hq=4, Hkv=2, Nq=64, Nk=64, d=64, causal=1,
             scale=0.125, odt=0)
    a.update(kw)
    return lib.attn_fwd_bias(a["q"], a["k"], a["v"], *_bias(a), a["o"], a["lse"], a["B"], a["Hq"], a["Hkv"],
                             a["Nq"], a["Nk"], a["d"], a["causal"], a["scale"], a["odt"], None, 0, None)


@pytest.mark.parametrize("kw,code", BAD_BIAS + [
    (dict(q=None), 1), (dict(v=FAKE + 8), 1), (dict(o=None), 1), (dict(lse=FAKE + 2), 1), (dict(Hq=3), 1),
    (dict(Nq=65), 1), (dict(Nq=0), 1), (dict(causal=2), 1), (dict(scale=-1.0), 1), (dict(odt=7), 1)])
def test_forward_refusals(lib, kw, code):
    assert fwd(lib, **kw) == code


def varlen(lib, **kw):
    a = dict(BIAS, q=FAKE, k=FAKE, v=FAKE, o=FAKE, cq=FAKE, ck=FAKE, B=2, Hq=4, Hkv=2, tq=100, tk=100, mq=64, mk=64,
             d=64, causal=1, scale=0.125, odt=0)
    a.update(kw)
    return lib.attn_fwd_varlen_bias(a["q"], a["k"], a["v"], *_bias(a), a["o"], None, a["cq"], a["ck"], a["B"],
                                    a["Hq"], a["Hkv"], a["tq"], a["tk"], a["mq"], a["mk"], a["d"], a["causal"],
                                    a["scale"], a["odt"], None)


@pytest.mark.parametrize("kw,code", BAD_BIAS + [
    (dict(cq=None), 1), (dict(ck=FAKE + 1), 1), (dict(tq=0), 1), (dict(mq=101), 1), (dict(mk=0), 1),
    (dict(causal=-1), 1)])
def test_packed_forward_refusals(lib, kw, code):
    assert varlen(lib, **kw) == code


def bwd(lib, packed, **kw):
    a = dict(BIAS, q=FAKE, o=FAKE, do=FAKE, lse=FAKE, dq=FAKE, dk=FAKE, dt=FAKE, cq=FAKE, Hq=4, d=64, gt=0, ws=FAKE,
             wsb=1 << 40, n=64, B=1, m=64)
    a.update(kw)
    head = (a["q"], FAKE, FAKE, a["o"], a["do"], a["lse"], *_bias(a), a["dq"], a["dk"], FAKE, a["dt"])
    if packed:
        return lib.attn_bwd_varlen_bias(*head, a["cq"], FAKE, 1, a["Hq"], 2, 64, 64, a["n"], 64, a["d"], 1, 0.125, 0,
                                        a["gt"], a["ws"], a["wsb"], None)
    return lib.attn_bwd_bias(*head, a["B"], a["Hq"], 2, a["n"], a["m"], a["d"], 1, 0.125, 0, a["gt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kw,code", BAD_BIAS + [
    (dict(q=None), 1), (dict(do=None), 1), (dict(lse=None), 1), (dict(dq=FAKE + 8), 1), (dict(dk=None), 1),
    (dict(dt=None), 1), (dict(dt=FAKE + 2), 1), (dict(gt=3), 1), (dict(Hq=65536), 2), (dict(Hq=5), 1), (dict(n=65), 1),
    (dict(ws=None), 5), (dict(wsb=64), 5), (dict(ws=FAKE + 8), 5)])
def test_backward_refusals(lib, packed, kw, code):
    assert bwd(lib, packed, **kw) == code


def test_backward_workspace(lib):
    base = ea.attn_bwd_workspace_size(2, 4, 2, 100, 300, 64)
    assert ea.attn_bwd_bias_workspace_size(2, 4, 2, 100, 300, 64, 114) == base + 16 + 4 * 4 * 132 * (6 + 1)
    assert ea.attn_bwd_bias_workspace_size(200, 1, 1, 100, 300, 64, 1) == \
        ea.attn_bwd_workspace_size(200, 1, 1, 100, 300, 64) + 16 + 4 * 20 * (600 + 2)
    assert ea.attn_bwd_varlen_bias_workspace_size(2, 4, 2, 100, 300, 64, 114) == \
        ea.attn_bwd_varlen_workspace_size(2, 4, 2, 100, 64) + 16 + 4 * 4 * 132 * (6 + 1)
    assert ea.attn_bwd_varlen_bias_workspace_size(1 << 13, 1, 1, 100, 1 << 24, 64, 1) > 0
    assert ea.attn_bwd_varlen_bias_workspace_size((1 << 13) + 1, 1, 1, 100, 1 << 24, 64, 1) == 0
    assert ea.attn_bwd_bias_workspace_size((1 << 13) + 1, 1, 1, 100, 1 << 24, 64, 1) == 0
    assert bwd(lib, False, B=(1 << 13) + 1, m=1 << 24) == 2
    for bad in (dict(d=136), dict(span=0), dict(span=65537), dict(Hq=3), dict(Hq=131072)):
        a = dict(Hq=4, d=64, span=114)
        a.update(bad)
        assert ea.attn_bwd_bias_workspace_size(2, a["Hq"], 2, 100, 300, a["d"], a["span"]) == 0
        assert ea.attn_bwd_varlen_bias_workspace_size(2, a["Hq"], 2, 100, 300, a["d"], a["span"]) == 0


def decode(lib, **kw):
    a = dict(BIAS, q=FAKE, kp=FAKE, bt=FAKE, sl=FAKE, o=FAKE, Hq=4, nb_pages=10, page=64, mb=4, d=64, scale=0.125,
             splits=0)
    a.update(kw)
    return lib.attn_decode_paged_bias(a["q"], a["kp"], FAKE, a["bt"], a["sl"], *_bias(a), a["o"], None, 2, a["Hq"],
                                      2, a["nb_pages"], a["page"], a["mb"], a["d"], a["scale"], a["splits"], FAKE,
                                      1 << 40, 0, None)


@pytest.mark.parametrize("kw,code", BAD_BIAS + [
    (dict(q=None), 1), (dict(kp=FAKE + 4), 1), (dict(bt=None), 1), (dict(sl=None), 1), (dict(o=None), 1),
    (dict(page=32), 1), (dict(page=96), 2), (dict(mb=0), 1), (dict(nb_pages=0), 1), (dict(Hq=34), 2),
    (dict(splits=-1), 1), (dict(scale=math.inf), 1)])
def test_decode_refusals(lib, kw, code):
    assert decode(lib, **kw) == code


def extend(lib, **kw):
    a = dict(pool=FAKE, blocks=100, bt=FAKE, sl=FAKE, new=FAKE, slots=FAKE, pos=2 * FAKE, cu=2 * FAKE,
             granted=2 * FAKE, B=4, mb=8, page=16, width=0, total=50)
    a.update(kw)
    return lib.attn_pages_extend(a["pool"], a["blocks"], a["bt"], a["sl"], a["new"], a["slots"], a["pos"], a["cu"],
                                 a["granted"], a["B"], a["mb"], a["page"], a["width"], a["total"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(pool=None), 1), (dict(pool=FAKE + 4), 1), (dict(bt=None), 1), (dict(sl=None), 1), (dict(new=FAKE + 1), 1),
    (dict(slots=None), 1), (dict(slots=FAKE + 8), 1), (dict(pos=2 * FAKE + 4), 1), (dict(cu=2 * FAKE + 2), 1),
    (dict(granted=2 * FAKE + 2), 1), (dict(blocks=0), 1),
    (dict(new=3 * FAKE, granted=3 * FAKE), 1), (dict(sl=3 * FAKE, cu=3 * FAKE), 1), (dict(B=0), 1), (dict(mb=0), 1), (dict(page=0), 1),
    (dict(width=-1), 1), (dict(total=-1), 1), (dict(width=3), 1), (dict(width=3, total=0), 1),
    (dict(width=1 << 29, total=0, cu=None), 1), (dict(mb=1 << 20, page=32), 1), (dict(blocks=(1 << 30) + 1), 2)])
def test_extend_refusals(lib, kw, code):
    assert extend(lib, **kw) == code


@pytest.mark.parametrize("at,value", [(0, None), (0, FAKE + 4), (2, None), (3, None), (4, None), (1, 0), (5, 0), (6, 0),
                                      (7, 0)])
def test_trim_refusals(lib, at, value):
    args = [FAKE, 100, FAKE, FAKE, FAKE, 4, 8, 16, None]
    args[at] = value
    assert lib.attn_pages_trim(*args) == 1


def test_pool_refusals(lib):
    assert lib.attn_page_pool_init(None, 4, None) == 1 and lib.attn_page_pool_init(FAKE + 4, 4, None) == 1
    assert lib.attn_page_pool_init(FAKE, 0, None) == 1 and lib.attn_page_pool_init(FAKE, (1 << 30) + 1, None) == 2


@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("n,D", [(32, 128), (8, 20), (4, 5), (64, 1000), (128, 2048), (16, 16384), (6, 7), (256, 4000)])
def test_buckets(n, D, both):
    buckets, first = ea.attn_bias_buckets(n, D, both)
    side = n // 2 if both else n
    assert buckets[-first] == 0 and buckets[0] == side - 1 and buckets[1] < side - 1
    assert [buckets[-first - r] for r in range(-first + 1)] == [bucket(r, side, D) for r in range(-first + 1)]
    assert buckets[-first + 1:] == ([side + bucket(r, side, D) for r in range(1, -first + 1)] if both else [])


def test_bucket_borders_are_exact():
    """Where e (D / e)^(k / s) is a whole number, the distance itself is in the new bucket: 8 * 2^(k / 2)."""
    buckets, first = ea.attn_bias_buckets(32, 128, True)
    for k, r in enumerate((8, 16, 32, 64)):
        assert buckets[-first - r] == 8 + 2 * k and buckets[-first - r + 1] == 7 + 2 * k
        assert buckets[-first + r] == 24 + 2 * k


def test_bucket_refusals(lib):
    i, n = ctypes.c_int(), ctypes.c_int()
    out = (ctypes.c_int * 200)()

    def call(*a, buckets=None, capacity=0, first=ctypes.byref(i)):
        return lib.attn_bias_buckets(*a, buckets, capacity, first, ctypes.byref(n))
    assert call(1, 128, 0) == 1 and call(2, 128, 1) == 1 and call(33, 128, 1) == 1
    assert call(32, 16, 0) == 1 and call(32, 8, 1) == 1 and call(32, 128, 2) == 1
    assert call(32, 128, 0, first=None) == 1
    assert call(1026, 1 << 20, 0) == 2 and call(32, 1 << 25, 0) == 2 and call(32, 1 << 23, 0) == 2
    assert call(32, 128, 0, buckets=out, capacity=113) == 1 and n.value == 114
    assert call(32, 128, 0, buckets=out, capacity=114) == 0 and out[113] == 0 and out[0] == 31


def test_python_refusals():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ea.attn_fwd_bias(x, x, x, torch.zeros(4, 2), torch.zeros(3, dtype=torch.int32), 0, x)
    with pytest.raises(ValueError, match="either width or total"):
        ea.pages_extend(None, None, torch.zeros(2), None, 16)
    with pytest.raises(ValueError, match="either width or total"):
        ea.pages_extend(None, None, torch.zeros(2), None, 16, width=1, total=3)


def test_reference_against_autograd():
    """The tests' own 64-bit gradients, the table's among them."""
    g = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(h, 7, 8, generator=g) for h in (4, 2, 2, 4))
    ids, t = torch.tensor([2, 0, 1, 1, 0], dtype=torch.int32), torch.randn(3, 4, generator=g)
    ref = Problem(q, k, v, t, ids, -3, True)
    leaves = [x.double().requires_grad_() for x in (q, k, v, t)]
    r = torch.arange(7) - torch.arange(7)[:, None]
    kk, vv = (x.repeat_interleave(2, 0) for x in leaves[1:3])
    x = leaves[0] @ kk.transpose(1, 2) / 8 ** 0.5 + leaves[3].t()[:, ids.long()[(r + 3).clamp(0, 4)]]
    o = x.masked_fill(torch.ones(7, 7).triu(1).bool(), -math.inf).softmax(-1) @ vv
    (o * do.double()).sum().backward()
    assert torch.allclose(o, ref.o, atol=1e-12)
    for got, leaf in zip(ref.gradients(ref.o, do, ref.lse, 3)[0], leaves):
        assert torch.allclose(got, leaf.grad, atol=1e-12)


def test_reference_pages():
    """The tests' own tables: pages in order, whole requests, nothing after the pool ran out."""
    p = Pages(5, 4, 9, 4)
    assert p.extend([5, 0, 9, 1]) == [([0, 1, 2, 3, 4], [0, 1, 2, 3, 4], 5), ([], [], 0),
                                      ([8 + i for i in range(9)], list(range(9)), 9), ([-1], [0], 0)]
    assert p.extend([3, 1, 0, 0])[0] == ([5, 6, 7], [5, 6, 7], 3) and p.len == [8, 0, 9, 0]
    p.trim([1, 0, 0, 0])
    assert p.free == [4, 3, 2, 1] and p.len == [1, 0, 0, 0]
