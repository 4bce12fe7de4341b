"""Attention with a learned relative position bias where a block of the persistent kernels
takes several work items: forward, packed forward and gradients against 64 bits, all outputs
(the items off a list, the windows and the diagonals' sums run on from one into the next).
In the dense calls an item's key tiles are odd in number, so that what is held twice starts
each item on the other half."""
import pytest
import torch

import exact_attention_14_gb300 as ea
from bias_ref import Problem, check_gradients

pytestmark = pytest.mark.gpu

MAPS = ["two-way", "long"]     # most tiles beyond the map, and all of them inside


def _map(kind):
    return *(ea.attn_bias_buckets(32, 128, True) if kind == "two-way" else ea.attn_bias_buckets(64, 700, True)),


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _inputs(Hq, Hkv, n, m, d, nb, seed):
    g = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g).to(torch.bfloat16)
    return (randn(Hq, n, d), randn(Hkv, m, d), randn(Hkv, m, d), randn(Hq, n, d),
            torch.randn(nb, Hq, generator=g) * 2)


def _by_group(q, k, v, table, ids, first, causal):
    """A Problem for each KV head, with the slice of its query heads."""
    G = q.shape[0] // k.shape[0]
    for h in range(k.shape[0]):
        at = slice(h * G, (h + 1) * G)
        yield h, at, Problem(q[at], k[h:h + 1], v[h:h + 1], table[:, at], ids, first, causal)


@pytest.mark.parametrize("kind", MAPS)
@pytest.mark.parametrize("d,causal", [(128, False), (128, True), (96, True), (64, False), (64, True)])
def test_forward(d, causal, kind):
    Hq, Hkv, n, m = 160, 32, 600, 600
    assert Hq * -(-n // 256) > 3 * _sms()
    buckets, first = _map(kind)
    ids = torch.tensor(buckets, dtype=torch.int32)
    q, k, v, _, table = _inputs(Hq, Hkv, n, m, d, 64, seed=d)
    o, lse = ea.forward_bias(q[None].cuda(), k[None].cuda(), v[None].cuda(), table.cuda(), ids.cuda(), first,
                             causal=causal)
    assert ea.attn_last_device_error() == 0
    o, lse = o[0].cpu(), lse[0].cpu()
    for _, at, ref in _by_group(q, k, v, table, ids, first, causal):
        ref.check_forward(o[at], lse[at])


@pytest.mark.parametrize("kind", MAPS)
@pytest.mark.parametrize("Hq,d,causal", [(96, 128, False), (96, 128, True), (192, 80, True), (96, 64, True)])
def test_gradients(Hq, d, causal, kind):
    Hkv, n, m = 96, 570, 600
    assert Hkv * -(-m // 128) > 3 * _sms() and Hq * -(-n // 128) > 3 * _sms()
    buckets, first = _map(kind)
    ids = torch.tensor(buckets, dtype=torch.int32)
    q, k, v, dout, table = _inputs(Hq, Hkv, n, m, d, 64, seed=d + 1)
    qg, kg, vg, dg = (t[None].cuda() for t in (q, k, v, dout))
    tg, ig = table.cuda(), ids.cuda()
    o, lse = ea.forward_bias(qg, kg, vg, tg, ig, first, causal=causal)
    dq, dk, dv, dt = (t.cpu() for t in ea.backward_bias(qg, kg, vg, o, dg, lse, tg, ig, first, causal=causal))
    assert ea.attn_last_device_error() == 0
    o, lse = o[0].cpu(), lse[0].cpu()
    for h, at, ref in _by_group(q, k, v, table, ids, first, causal):
        ref.check_forward(o[at], lse[at])
        grads, bounds = ref.gradients(o[at], dout[at], lse[at], 64)
        check_gradients([dq[0, at], dk[0, h:h + 1], dv[0, h:h + 1], dt[:, at]], grads, bounds)


@pytest.mark.parametrize("kind", MAPS)
@pytest.mark.parametrize("d,causal", [(128, True), (128, False), (64, True)])
def test_packed(d, causal, kind):
    """Sequences of one row to several tiles, more keys than queries in some."""
    Hq = Hkv = 64
    nq, nk = [600, 1, 257, 500, 127, 300, 385], [600, 1, 300, 500, 129, 300, 600]
    assert Hkv * sum(-(-x // 128) for x in nk) > 3 * _sms() and Hq * sum(-(-x // 128) for x in nq) > 3 * _sms()
    assert Hq * sum(-(-x // 256) for x in nq) > 3 * _sms()
    buckets, first = _map(kind)
    ids = torch.tensor(buckets, dtype=torch.int32)
    q, k, v, dout, table = _inputs(Hq, Hkv, sum(nq), sum(nk), d, 64, seed=d + 2)
    cq, ck = (torch.tensor([0] + x).cumsum(0).to(torch.int32) for x in (nq, nk))
    qg, kg, vg, dg = (t.transpose(0, 1).contiguous().cuda() for t in (q, k, v, dout))
    tg, ig, at = table.cuda(), ids.cuda(), (cq.cuda(), ck.cuda(), max(nq), max(nk))
    o, lse = ea.forward_varlen_bias(qg, kg, vg, *at, tg, ig, first, causal=causal)
    got = ea.backward_varlen_bias(qg, kg, vg, o, dg, lse, *at, tg, ig, first, causal=causal)
    assert ea.attn_last_device_error() == 0
    o, lse = o.cpu().transpose(0, 1), lse.cpu()
    dq, dk, dv = (t.cpu().transpose(0, 1) for t in got[:3])
    want, bound = (torch.zeros(64, Hq, dtype=torch.float64) for _ in range(2))
    for b in range(len(nq)):
        x, y = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        for h in range(Hq):
            at = slice(h, h + 1)
            ref = Problem(q[at, x], k[at, y], v[at, y], table[:, at], ids, first, causal)
            ref.check_forward(o[at, x], lse[at, x])
            grads, bounds = ref.gradients(o[at, x], dout[at, x], lse[at, x], 64)
            want[:, at] += grads.pop()
            bound[:, at] += bounds.pop()
            check_gradients([dq[at, x], dk[at, y], dv[at, y]], grads, bounds)
    check_gradients([got[3]] * 4, [want] * 4, [bound] * 4)


def test_one_item_of_two_million_tiles():
    """A key tile whose 14 heads of 2^24 queries all lie past the map: the warp that adds up
    distances has nothing to do and waits over 2 s, a wait's bound, for the next item.  Queries
    of zeros, keys, values, O and dO of ones: P is 1/8, dS 0.  dV is a sum of 14 * 2^24 eighths
    in fp32: exact below 2^21, where fp32's step is at most 1/8; from there on an addend may be
    lost but none is added twice, so it ends between 2^21 and 14 * 2^21."""
    H, n, m, d = 14, 1 << 24, 8, 8
    ones = torch.ones(1, H, n, d, dtype=torch.bfloat16, device="cuda")
    q, dq = torch.zeros_like(ones), torch.empty_like(ones)
    k = torch.ones(1, 1, m, d, dtype=torch.bfloat16, device="cuda")
    dk, dv = torch.empty_like(k), torch.empty_like(k)
    lse = torch.full((1, H, n), 8.0, device="cuda").log_()
    ids, table = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, H, device="cuda")
    dtable = torch.empty_like(table)
    ea.attn_bwd_bias(q, k, k, ones, ones, lse, table, ids, -1000, dq, dk, dv, dtable)
    assert ea.attn_last_device_error() == 0
    assert (dv >= 2 ** 21).all() and (dv <= H * 2 ** 21).all()
    assert not dk.any() and not dtable.any() and not dq.any()
