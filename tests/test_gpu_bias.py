"""Attention with a learned relative position bias against 64 bits: forward,
gradients and paged decode, at the sizes, maps and tables where they can go
wrong.  Bounds element by element, from the roundings (bias_ref)."""
import math

import pytest
import torch

import exact_attention_14_gb300 as ea
from bias_ref import Problem, check_gradients

pytestmark = pytest.mark.gpu


def _inputs(B, Hq, Hkv, n, m, d, seed=0):
    g = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g).to(torch.bfloat16)
    return randn(B, Hq, n, d), randn(B, Hkv, m, d), randn(B, Hkv, m, d), randn(B, Hq, n, d), g


def _map(kind, g):
    """(buckets, first, how many buckets)"""
    if kind == "two-way":
        return *ea.attn_bias_buckets(32, 128, True), 32
    if kind == "one-way":
        return *ea.attn_bias_buckets(32, 128, False), 32
    if kind == "long":
        return *ea.attn_bias_buckets(64, 700, True), 64
    if kind == "scrambled":         # any map will do: no order, some buckets unused
        return torch.randint(0, 17, (301,), generator=g).tolist(), -140, 19
    if kind == "one distance":      # every tile has one bias
        return [3], 5, 4
    if kind == "only ahead":        # the whole map lies after the query
        return list(range(40)), 7, 40
    if kind == "far back":
        return list(range(33)), -400, 33
    raise AssertionError(kind)


def _table(g, nb, Hq, dtype=torch.float32):
    return (torch.randn(nb, Hq, generator=g) * 2).to(dtype)


def _gpu(*ts):
    return [t.cuda() for t in ts]


SHAPES = [  # B, Hq, Hkv, n, m, d, causal
    (1, 1, 1, 1, 1, 64, False), (1, 2, 1, 1, 300, 128, True), (2, 4, 2, 129, 129, 64, True),
    (1, 3, 3, 200, 333, 72, False), (2, 2, 1, 127, 640, 128, True), (1, 4, 4, 513, 511, 128, False),
    (1, 2, 2, 384, 1000, 16, False), (1, 6, 2, 700, 700, 96, True),
]
MAPS = ["two-way", "one-way", "long", "scrambled", "one distance", "only ahead", "far back"]


@pytest.mark.parametrize("kind", MAPS)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, kind):
    B, Hq, Hkv, n, m, d, causal = shape
    q, k, v, _, g = _inputs(B, Hq, Hkv, n, m, d)
    buckets, first, nb = _map(kind, g)
    out32 = kind in ("one-way", "scrambled")
    table = _table(g, nb, Hq, torch.bfloat16 if kind in ("long", "scrambled") else torch.float32)
    ids = torch.tensor(buckets, dtype=torch.int32)
    o, lse = ea.forward_bias(*_gpu(q, k, v, table, ids), first, causal=causal,
                             out_dtype=torch.float32 if out32 else torch.bfloat16)
    assert ea.attn_last_device_error() == 0
    for b in range(B):
        Problem(q[b], k[b], v[b], table, ids, first, causal).check_forward(o[b], lse[b])


def test_forward_split_tail():
    """Non-causal shapes whose last units are cut along the keys: the merge meets rows
    that have no key in a piece (a bias of -inf) and rows that have none at all."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    B, Hq, n, m, d = 1, 2, 300, 1500, 128
    full, split, parts = ea.attn_fwd_split_plan(B, Hq, Hq, n, m, d, False, sms)
    assert split > 0 and parts > 1
    q, k, v, _, g = _inputs(B, Hq, Hq, n, m, d)
    buckets = list(range(50))
    ids = torch.tensor(buckets, dtype=torch.int32)
    table = _table(g, 50, Hq)
    for o_type in (torch.bfloat16, torch.float32):
        o, lse = ea.forward_bias(*_gpu(q, k, v, table, ids), -1000, out_dtype=o_type)
        Problem(q[0], k[0], v[0], table, ids, -1000).check_forward(o[0], lse[0])
    table[0, 0] = -math.inf             # head 0: only keys less than 1000 back
    table[20:, 1] = -math.inf           # head 1: keys at least 981 back; for the first rows none
    o, lse = ea.forward_bias(*_gpu(q, k, v, table, ids), -1000)
    ref = Problem(q[0], k[0], v[0], table, ids, -1000)
    ref.check_forward(o[0], lse[0])
    table[:] = torch.finfo(torch.float32).min
    table[:, 1] = 0.5
    o, lse = ea.forward_bias(*_gpu(q, k, v, table, ids), -1000)
    assert (o[0, 0] == 0).all() and (lse[0, 0] == -math.inf).all()
    Problem(q[0], k[0], v[0], table, ids, -1000).check_forward(o[0], lse[0])


@pytest.mark.parametrize("low", [-math.inf, -1e9, torch.finfo(torch.float32).min, torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("causal", [False, True])
def test_masked_buckets(causal, low):
    """Buckets that leave their keys out: forward, gradients, rows without any key."""
    q, k, v, dout, g = _inputs(1, 4, 2, 260, 390, 64)
    buckets, first, nb = _map("two-way", g)
    ids = torch.tensor(buckets, dtype=torch.int32)
    table = _table(g, nb, 4)
    table[15, 0] = table[31, 0] = low   # head 0 sees less than 113 positions
    table[:14, 1] = low                 # head 1 sees far keys only (causal: some rows none)
    table[16:, 1] = low
    table[:, 2] = low                   # head 2 sees nothing
    qg, kg, vg, tg, ig, dg = _gpu(q, k, v, table, ids, dout)
    o, lse = ea.forward_bias(qg, kg, vg, tg, ig, first, causal=causal, out_dtype=torch.float32)
    ref = Problem(q[0], k[0], v[0], table, ids, first, causal)
    assert (ref.lse[2] == -math.inf).all()
    ref.check_forward(o[0], lse[0])
    got = ea.backward_bias(qg, kg, vg, o, dg, lse, tg, ig, first, causal=causal, grad_dtype=torch.float32)
    grads, bounds = ref.gradients(o[0], dout[0], lse[0], nb)
    check_gradients([got[0][0], got[1][0], got[2][0], got[3]], grads, bounds)
    assert (got[3][:, 2] == 0).all() and (got[0][0, 2] == 0).all()


@pytest.mark.parametrize("by", [9.99e5, -9.99e5])
def test_large_biases_stay_finite(by):
    """All biases near the largest allowed: O and LSE hold (scores keep 2^-4 there), gradients are finite."""
    q, k, v, dout, g = _inputs(1, 2, 2, 200, 200, 64)
    ids, table = torch.arange(9, dtype=torch.int32), torch.full((9, 2), by)
    qg, kg, vg, tg, ig, dg = _gpu(q, k, v, table, ids, dout)
    o, lse = ea.forward_bias(qg, kg, vg, tg, ig, -4)
    assert (lse - by).abs().max() < 16 and torch.isfinite(o.float()).all()
    for x in ea.backward_bias(qg, kg, vg, o, dg, lse, tg, ig, -4):
        assert torch.isfinite(x.float()).all()


@pytest.mark.parametrize("kind", MAPS)
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients(shape, kind):
    B, Hq, Hkv, n, m, d, causal = shape
    q, k, v, dout, g = _inputs(B, Hq, Hkv, n, m, d, seed=1)
    buckets, first, nb = _map(kind, g)
    ids = torch.tensor(buckets, dtype=torch.int32)
    table = _table(g, nb, Hq, torch.bfloat16 if kind in ("long", "scrambled") else torch.float32)
    qg, kg, vg, tg, ig, dg = _gpu(q, k, v, table, ids, dout)
    o, lse = ea.forward_bias(qg, kg, vg, tg, ig, first, causal=causal)
    gt = torch.float32 if kind in ("one-way", "scrambled") else torch.bfloat16
    got = ea.backward_bias(qg, kg, vg, o, dg, lse, tg, ig, first, causal=causal, grad_dtype=gt)
    assert ea.attn_last_device_error() == 0
    want = None
    for b in range(B):
        grads, bounds = Problem(q[b], k[b], v[b], table, ids, first, causal).gradients(o[b], dout[b], lse[b], nb)
        check_gradients([got[0][b], got[1][b], got[2][b]], grads[:3], bounds[:3])
        want = (grads[3], bounds[3]) if want is None else (want[0] + grads[3], want[1] + bounds[3])
    check_gradients([got[3]] * 4, [want[0]] * 4, [want[1]] * 4)
    again = ea.backward_bias(qg, kg, vg, o, dg, lse, tg, ig, first, causal=causal, grad_dtype=gt)
    assert all(torch.equal(a, b) for a, b in zip(got, again))      # bit for bit


def test_gradient_is_the_slope():
    """dtable against central differences of sum(O dO) in the forward's fp32 output:
    a step of 2^-3 along a direction, the truncation (step^2 times a third derivative
    at most 6 max |O dO| n) and twice the forward's own error as the bound."""
    B, H, n, d = 1, 2, 130, 64
    q, k, v, dout, g = _inputs(B, H, H, n, n, d, seed=3)
    buckets, first, nb = _map("two-way", g)
    ids = torch.tensor(buckets, dtype=torch.int32)
    table, along = _table(g, nb, H), torch.randn(nb, H, generator=g) * 2.0 ** -3
    o, lse = ea.forward_bias(*_gpu(q, k, v, table, ids), first, out_dtype=torch.float32)
    *_, dtable = ea.backward_bias(*_gpu(q, k, v), o, dout.cuda(), lse, *_gpu(table, ids), first)

    def value(t):
        p = Problem(q[0], k[0], v[0], t, ids, first)
        return (p.o * dout[0].double()).sum()
    h = 2.0 ** -4
    slope = (value(table.double() + h * along.double()) - value(table.double() - h * along.double())) / (2 * h)
    fine = (value(table.double() + h / 2 * along.double()) - value(table.double() - h / 2 * along.double())) / h
    ref = Problem(q[0], k[0], v[0], table, ids, first)
    bounds = ref.gradients(o[0], dout[0], lse[0], nb)[1][3]
    # Richardson: the truncation left in `fine` is a third of the change, up to fourth order
    got = (dtable.cpu().double() * along).sum()
    # (D comes from O, whose weights were rounded to bf16: sum dS over a row is then off by |dO| |O - O64|)
    from_o = ((o[0].cpu().double() - ref.o).abs() * dout[0].double().abs()).sum(-1).sum() * along.abs().max()
    assert abs(got - fine) <= (bounds * along.abs()).sum() + (slope - fine).abs() + from_o


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,kind", [(64, "two-way"), (128, "long"), (80, "scrambled")])
def test_packed(d, kind, causal):
    """Packed batches with empty sequences, one-row ones, and rows that no sequence has."""
    lens_q, lens_k = [5, 0, 300, 1, 0, 129], [70, 0, 300, 1, 9, 400]
    Hq, Hkv = 4, 2
    cu_q = torch.tensor([2] + lens_q).cumsum(0).to(torch.int32)
    cu_k = torch.tensor([0] + lens_k).cumsum(0).to(torch.int32)
    tq, tk = int(cu_q[-1]) + 3, int(cu_k[-1])
    g = torch.Generator().manual_seed(4)
    q, dout = (torch.randn(tq, Hq, d, generator=g).to(torch.bfloat16) for _ in range(2))
    k, v = (torch.randn(tk, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    buckets, first, nb = _map(kind, g)
    ids, table = torch.tensor(buckets, dtype=torch.int32), _table(g, nb, Hq)
    qg, kg, vg, cq, ck, tg, ig, dg = _gpu(q, k, v, cu_q, cu_k, table, ids, dout)
    o = torch.full((tq, Hq, d), 7.0, device="cuda")
    lse = torch.full((Hq, tq), 7.0, device="cuda")
    ea.attn_fwd_varlen_bias(qg, kg, vg, tg, ig, first, o, cq, ck, 300, 400, lse, causal=causal)
    assert (o[:2] == 7).all() and (o[-3:] == 7).all() and (lse[:, :2] == 7).all() and (lse[:, -3:] == 7).all()
    grads = [torch.full(s, 7.0, device="cuda") for s in (q.shape, k.shape, v.shape, table.shape)]
    ea.attn_bwd_varlen_bias(qg, kg, vg, o, dg, lse, tg, ig, first, *grads, cq, ck, 300, 400, causal=causal)
    assert ea.attn_last_device_error() == 0
    assert (grads[0][:2] == 7).all() and (grads[0][-3:] == 7).all()
    total = [torch.zeros(nb, Hq, dtype=torch.float64) for _ in range(2)]
    for b in range(6):
        i0, i1, j0, j1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        if i0 == i1:
            assert (grads[1][j0:j1] == 0).all() and (grads[2][j0:j1] == 0).all()
            continue

        def part(t, a, z):
            return t[a:z].transpose(0, 1)
        ref = Problem(part(q, i0, i1), part(k, j0, j1), part(v, j0, j1), table, ids, first, causal)
        ref.check_forward(part(o, i0, i1), lse[:, i0:i1])
        want, bounds = ref.gradients(part(o, i0, i1), part(dout, i0, i1), lse[:, i0:i1], nb)
        check_gradients([part(grads[0], i0, i1), part(grads[1], j0, j1), part(grads[2], j0, j1)], want[:3], bounds[:3])
        total[0] += want[3]
        total[1] += bounds[3]
    check_gradients([grads[3]] * 4, [total[0]] * 4, [total[1]] * 4)


def test_many_key_tiles():
    """More than 512 key tiles in a batch: their sums are added by several blocks."""
    q, k, v, dout, g = _inputs(200, 1, 1, 130, 257, 8, seed=5)
    ids, table = torch.tensor(list(range(61)), dtype=torch.int32), _table(g, 61, 1)
    qg, kg, vg, tg, ig, dg = _gpu(q, k, v, table, ids, dout)
    o, lse = ea.forward_bias(qg, kg, vg, tg, ig, -30)
    got = ea.backward_bias(qg, kg, vg, o, dg, lse, tg, ig, -30)
    want = torch.zeros(61, 1, dtype=torch.float64), torch.zeros(61, 1, dtype=torch.float64)
    for b in range(200):
        grads, bounds = Problem(q[b], k[b], v[b], table, ids, -30).gradients(o[b], dout[b], lse[b], 61)
        want[0].add_(grads[3])
        want[1].add_(bounds[3])
    check_gradients([got[3]] * 4, [want[0]] * 4, [want[1]] * 4)


def test_zero_bias_and_zero_scale():
    """A table of one zero is plain attention, whose outputs keep the same bounds; scale 0
    leaves softmax(bias)."""
    q, k, v, _, g = _inputs(1, 2, 2, 300, 384, 128, seed=6)
    ids = torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 2)
    for causal in (False, True):
        ref = Problem(q[0], k[0], v[0], table, ids, 0, causal)
        for o, lse in (ea.forward_bias(*_gpu(q, k, v, table, ids), 0, causal=causal),
                       ea.forward(*_gpu(q, k, v), causal=causal)):
            ref.check_forward(o[0], lse[0])
    buckets, first, nb = _map("two-way", g)
    ids, table = torch.tensor(buckets, dtype=torch.int32), _table(g, nb, 2)
    o, lse = ea.forward_bias(*_gpu(q, k, v, table, ids), first, scale=0.0)
    Problem(q[0], k[0], v[0], table, ids, first, scale=0.0).check_forward(o[0], lse[0])


def test_large_biases():
    """Biases far below and above the scores: rows whose logsumexp leaves 2^+-128, keys
    past the last one included (their 2^-lse must not reach dQ)."""
    q, k, v, dout, g = _inputs(1, 2, 2, 70, 197, 64, seed=7)
    buckets, first, nb = _map("two-way", g)
    ids = torch.tensor(buckets, dtype=torch.int32)
    for offset in (-3000.0, 3000.0):
        table = _table(g, nb, 2) + offset
        qg, kg, vg, tg, ig, dg = _gpu(q, k, v, table, ids, dout)
        o, lse = ea.forward_bias(qg, kg, vg, tg, ig, first, out_dtype=torch.float32)
        ref = Problem(q[0], k[0], v[0], table, ids, first)
        ref.check_forward(o[0], lse[0])
        got = ea.backward_bias(qg, kg, vg, o, dg, lse, tg, ig, first)
        grads, bounds = ref.gradients(o[0], dout[0], lse[0], nb)
        # (the weights follow from an lse that is itself off by its bound, for all of a row alike)
        slack = 2 * (ref.lse - lse[0].cpu().double()).abs().max() + 4 * ref.dx.max()
        bounds = [x + slack * y.abs() for x, y in zip(bounds, grads)]
        check_gradients([got[0][0], got[1][0], got[2][0], got[3]], grads, bounds)


@pytest.mark.parametrize("nb,kind", [(2400, "a distance each"), (1025, "runs"), (40000, "scrambled"), (1 << 16, "one")])
def test_many_buckets(nb, kind):
    """The table's gradient where a block has 64 buckets, and several heads one after the other."""
    q, k, v, dout, g = _inputs(1, 6, 3, 200, 330, 64, seed=nb)
    if kind == "a distance each":
        ids, first = torch.arange(nb, dtype=torch.int32), -1300
    elif kind == "runs":
        ids, first = torch.arange(3000, dtype=torch.int32) // 3 + 25, -1500
    elif kind == "scrambled":
        ids, first = torch.randint(0, nb, (900,), generator=g, dtype=torch.int32), -400
        ids[::7] = nb - 1
    else:
        ids, first = torch.full((300,), nb - 1, dtype=torch.int32), -100
    table = _table(g, nb, 6)
    o, lse = ea.forward_bias(*_gpu(q, k, v, table, ids), first)
    ref = Problem(q[0], k[0], v[0], table, ids, first)
    ref.check_forward(o[0], lse[0])
    got = ea.backward_bias(*_gpu(q, k, v), o, dout.cuda(), lse, *_gpu(table, ids), first, grad_dtype=torch.float32)
    grads, bounds = ref.gradients(o[0], dout[0], lse[0], nb)
    check_gradients([got[0][0], got[1][0], got[2][0], got[3]], grads, bounds)
    used = torch.zeros(nb, dtype=torch.bool)
    used[ids.long()] = True
    assert (got[3].cpu()[~used] == 0).all()


def test_wrong_buckets_are_reported():
    q, k, v, dout, g = _inputs(1, 2, 2, 40, 40, 64)
    ids = torch.tensor([0, 5, 1], dtype=torch.int32)          # bucket 5 of 3: adds nothing
    table = _table(g, 3, 2)
    o, lse = ea.forward_bias(*_gpu(q, k, v, table, ids), -1)
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert ea.attn_last_device_error() == 0
    clean = torch.cat([table, torch.zeros(1, 2)])
    Problem(q[0], k[0], v[0], clean, torch.tensor([0, 3, 1]), -1).check_forward(o[0], lse[0])
    *_, dtable = ea.backward_bias(*_gpu(q, k, v), o, dout.cuda(), lse, *_gpu(table, ids), -1)
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert torch.isfinite(dtable).all() and (dtable[2] == 0).all()


def _pages(lengths, Hkv, d, page, seed=0, spare=0.0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lengths]
    perm = torch.randperm(sum(need) + 2, generator=g).tolist()
    table = torch.full((len(lengths), max(max(need), 1)), 2 ** 30, dtype=torch.int32)
    kp, vp = (torch.full((sum(need) + 2, page, Hkv, d), math.nan, dtype=torch.bfloat16) for _ in range(2))
    ks, vs = [], []
    for b, n in enumerate(lengths):
        k, v = (torch.randn(n, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
        for i in range(need[b]):
            at = perm.pop()
            table[b, i] = at
            rows = min(page, n - i * page)
            kp[at, :rows], vp[at, :rows] = k[i * page:i * page + rows], v[i * page:i * page + rows]
        ks.append(k)
        vs.append(v)
    return kp, vp, table, torch.tensor(lengths, dtype=torch.int32), ks, vs, g


@pytest.mark.parametrize("kind", MAPS)
@pytest.mark.parametrize("lengths,Hq,Hkv,d,page,splits", [
    ([1], 1, 1, 64, 64, 0), ([63, 64, 65, 1], 8, 2, 128, 64, 0), ([700, 2000], 16, 1, 96, 128, 0),
    ([1500], 6, 6, 8, 64, 7), ([130, 3333], 4, 4, 128, 256, 3)])
def test_decode(lengths, Hq, Hkv, d, page, splits, kind):
    kp, vp, bt, sl, ks, vs, g = _pages(lengths, Hkv, d, page)
    q = torch.randn(len(lengths), Hq, 1, d, generator=g).to(torch.bfloat16)
    buckets, first, nb = _map(kind, g)
    ids = torch.tensor(buckets, dtype=torch.int32)
    table = _table(g, nb, Hq, torch.bfloat16 if kind == "long" else torch.float32)
    o, lse = ea.decode_paged_bias(*_gpu(q, kp, vp, bt, sl, table, ids), first, num_splits=splits,
                                  out_dtype=torch.float32 if kind == "long" else torch.bfloat16)
    assert ea.attn_last_device_error() == 0
    for b in range(len(lengths)):
        Problem(q[b], ks[b].transpose(0, 1), vs[b].transpose(0, 1), table, ids, first).check_forward(o[b], lse[b])


def test_decode_masked_and_empty():
    """Chunks and whole rows without a key, and a sequence of length 0."""
    kp, vp, bt, sl, ks, vs, g = _pages([3000, 100, 900], 2, 64, 64)
    q = torch.randn(3, 4, 1, 64, generator=g).to(torch.bfloat16)
    buckets, first, nb = _map("one-way", g)
    ids, table = torch.tensor(buckets, dtype=torch.int32), _table(g, nb, 4)
    table[31, 0] = -math.inf            # head 0 sees 113 keys
    table[:31, 1] = -math.inf           # head 1 sees the far ones only (sequence 1: none)
    table[:, 2] = torch.finfo(torch.float32).min
    o, lse = ea.decode_paged_bias(*_gpu(q, kp, vp, bt, sl, table, ids), first)
    assert ea.attn_last_device_error() == 0
    for b in range(3):
        Problem(q[b], ks[b].transpose(0, 1), vs[b].transpose(0, 1), table, ids, first).check_forward(o[b], lse[b])
    sl[1] = 0
    o, lse = ea.decode_paged_bias(*_gpu(q, kp, vp, bt, sl, table, ids), first)
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()


def test_decode_many_groups():
    """More (sequence, KV head) groups than the in-kernel merge counts: the second kernel."""
    B, H = 600, 7
    assert ea.attn_decode_kernel_launches(B, H, H, 128, 64, 2) == 2
    kp, vp, bt, sl, ks, vs, g = _pages([1 + b % 128 for b in range(B)], H, 64, 128)
    q = torch.randn(B, H, 1, 64, generator=g).to(torch.bfloat16)
    ids, table = torch.tensor(list(range(100)), dtype=torch.int32), _table(g, 100, H)
    table[70:, 3] = -math.inf
    o, lse = ea.decode_paged_bias(*_gpu(q, kp, vp, bt, sl, table, ids), -99, num_splits=2)
    for b in list(range(0, B, 37)) + [127, 128]:
        Problem(q[b], ks[b].transpose(0, 1), vs[b].transpose(0, 1), table, ids, -99).check_forward(o[b], lse[b])


def test_streams_and_graphs():
    """A training step on another stream, and captured and replayed on new inputs with an
    eager call between the replays."""
    q, k, v, dout, g = _inputs(1, 4, 2, 300, 300, 128, seed=8)
    buckets, first, nb = _map("two-way", g)
    ids, table = torch.tensor(buckets, dtype=torch.int32), _table(g, nb, 4)
    qg, kg, vg, tg, ig, dg = _gpu(q, k, v, table, ids, dout)

    def step(stream=None):
        o, lse = ea.forward_bias(qg, kg, vg, tg, ig, first, causal=True, stream=stream)
        return (o, lse, *ea.backward_bias(qg, kg, vg, o, dg, lse, tg, ig, first, causal=True, stream=stream))
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (9, 10):
        q2, k2, v2, d2, _ = _inputs(1, 4, 2, 300, 300, 128, seed=seed)
        for dst, src in ((qg, q2), (kg, k2), (vg, v2), (dg, d2), (tg, table + seed)):
            dst.copy_(src)
        graph.replay()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
    assert ea.attn_last_device_error() == 0


def test_two_calls_at_once():
    """Steps in flight on two streams, each with its own workspaces."""
    sets = []
    for seed in (11, 12):
        q, k, v, dout, g = _inputs(2, 4, 4, 640, 640, 64, seed=seed)
        buckets, first, nb = _map("long", g)
        sets.append((*_gpu(q, k, v, dout, torch.tensor(buckets, dtype=torch.int32), _table(g, nb, 4)), first))

    def step(s, stream):
        q, k, v, dout, ids, table, first = s
        o, lse = ea.forward_bias(q, k, v, table, ids, first, stream=stream)
        return (o, lse, *ea.backward_bias(q, k, v, o, dout, lse, table, ids, first, stream=stream))
    want = [step(s, None) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [step(s, st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
