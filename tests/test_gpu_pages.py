"""The paged cache's tables on the GPU against plain Python, and a serving and a
training run of the operators together."""
import math
import random

import pytest
import torch

import exact_attention_14_gb300 as ea
from bias_ref import Pages, Problem, check_gradients

pytestmark = pytest.mark.gpu


def _state(pages, B):
    pool = ea.page_pool(pages.num_blocks)
    table = torch.full((B, pages.max_blocks), -1, dtype=torch.int32, device="cuda")
    return pool, table, torch.zeros(B, dtype=torch.int32, device="cuda")


def _same(pages, pool, table, seqlens):
    assert seqlens.tolist() == pages.len
    n = len(pages.free)
    assert pool[:4].tolist() == [n, 0, 0, 0] and pool[4:4 + n].tolist() == pages.free
    for b, n in enumerate(pages.len):
        used = -(-n // pages.page)
        assert table[b, :used].tolist() == pages.table[b][:used]


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,page,max_blocks,blocks", [
    (1, 1, 50, 50), (1, 64, 9, 3), (5, 16, 20, 60), (33, 7, 11, 150), (300, 16, 40, 2500), (1025, 64, 3, 2000),
    (4096, 16, 2, 5000)])
def test_steps(B, page, max_blocks, blocks):
    """Prompts, single tokens, drafts, cuts: packed and padded in turn, the pool running out."""
    rng = random.Random(B)
    pages = Pages(blocks, B, max_blocks, page)
    pool, table, seqlens = _state(pages, B)
    for step in range(8):
        room = [max_blocks * page - n for n in pages.len]
        kind = step % 4
        most = {0: max_blocks * page // 2, 1: 1, 2: 5, 3: page + 1}[kind]
        new = [min(r, rng.randint(0 if kind else 1, max(1, most))) for r in room]
        if kind == 0 and step:
            new = [0 if rng.random() < 0.7 else x for x in new]
        if kind in (0, 3):
            total = sum(new) + rng.choice([0, 1, 6])
            slots, pos, cu, granted = ea.pages_extend(pool, table, seqlens, _int(new), page, total=total)
            want = pages.extend(new)
            flat = [x for row, _, _ in want for x in row]
            assert slots.tolist() == flat + [-1] * (total - len(flat))
            flat = [x for _, row, _ in want for x in row]
            assert pos.tolist() == flat + [0] * (total - len(flat))
            assert cu.tolist() == [0] + torch.tensor(new).cumsum(0).tolist()
        else:
            width = max(max(new), 1) + step % 3
            slots, pos, granted = ea.pages_extend(pool, table, seqlens, _int(new), page, width=width)
            want = pages.extend(new, width)
            assert slots.tolist() == [row + [-1] * (width - len(row)) for row, _, _ in want]
            assert pos.tolist() == [row + [0] * (width - len(row)) for _, row, _ in want]
        assert granted.tolist() == [x for _, _, x in want]
        _same(pages, pool, table, seqlens)
        keep = [rng.choice([0, n, n + 5, rng.randint(0, n), max(0, n - 1), -3]) if rng.random() < 0.5 else n
                for n in pages.len]
        ea.attn_pages_trim(pool, table, seqlens, _int(keep), page)
        pages.trim(keep)
        _same(pages, pool, table, seqlens)
    assert ea.attn_last_device_error() == 0


def test_taken_and_given_back():
    """A step undone leaves the pool as it was, to the order of its pages."""
    pool = ea.page_pool(100)
    table = torch.full((4, 30), -1, dtype=torch.int32, device="cuda")
    seqlens, new = _int([0, 0, 0, 0]), _int([17, 0, 300, 33])
    before = pool.clone()
    first = ea.pages_extend(pool, table, seqlens, new, 16, total=350)
    ea.attn_pages_trim(pool, table, seqlens, _int([0] * 4), 16)
    assert torch.equal(pool, before) and seqlens.tolist() == [0] * 4
    again = ea.pages_extend(pool, table, seqlens, new, 16, total=350)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_what_is_refused_on_the_device():
    """Lengths that cannot be, rows that are too short, and pages given back twice: reported,
    and the rest of the batch served."""
    pool = ea.page_pool(40)
    table = torch.full((5, 4), -1, dtype=torch.int32, device="cuda")
    seqlens = _int([0, -1, 0, 60, 3])
    table[3] = _int([36, 37, 38, 39])
    table[4, 0] = 35
    new = _int([5, 4, -2, 9, 6])       # request 3: 69 > 4 * 16 tokens
    slots, pos, granted = ea.pages_extend(pool, table, seqlens, new, 16, width=6)
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert granted.tolist() == [5, 0, 0, 0, 6] and seqlens.tolist() == [5, -1, 0, 60, 9]
    assert slots.tolist()[0] == [0, 1, 2, 3, 4, -1] and slots.tolist()[4] == [35 * 16 + 3 + i for i in range(6)]
    assert (slots[1:4] == -1).all() and (pos[1:4] == 0).all() and pool[0] == 39
    # a padded row that is too narrow
    _, _, granted = ea.pages_extend(pool, table, seqlens, _int([3, 0, 0, 0, 1]), 16, width=2)
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert granted.tolist() == [0, 0, 0, 0, 1]
    # packed rows for fewer tokens than there are: the rest are not written
    seqlens = _int([5, 0, 0, 60, 9])
    slots = torch.full((4,), 77, dtype=torch.int64, device="cuda")
    ea.attn_pages_extend(pool, table, seqlens, _int([2, 0, 0, 0, 7]), 16, slots[:3])
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert slots.tolist()[:2] == [5, 6] and slots[3] == 77
    # an entry of the table that names no page
    table[4, 1] = 1000
    seqlens = _int([0, 0, 0, 0, 20])
    slots, *_ = ea.pages_extend(pool, table, seqlens, _int([0, 0, 0, 0, 2]), 16, width=2)
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert slots.tolist()[4] == [-1, -1]
    # more pages than the cache has
    pool = ea.page_pool(40)
    before, seqlens = pool.clone(), _int([16, 0, 0, 0, 0])
    ea.attn_pages_trim(pool, table, seqlens, _int([0] * 5), 16)
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert torch.equal(pool, before) and seqlens.tolist() == [16, 0, 0, 0, 0]
    # a length the table cannot hold stays
    seqlens = _int([0, 0, 65, 0, -5])
    ea.attn_pages_trim(pool, table, seqlens, _int([0] * 5), 16)
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert torch.equal(pool, before) and seqlens.tolist() == [0, 0, 65, 0, -5]


def test_no_tokens_at_all():
    pool = ea.page_pool(3)
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    seqlens = _int([0, 0])
    slots, pos, cu, granted = ea.pages_extend(pool, table, seqlens, _int([0, 0]), 16, total=0)
    assert slots.numel() == 0 and cu.tolist() == [0, 0, 0] and granted.tolist() == [0, 0]
    assert pool.tolist() == [3, 0, 0, 0, 2, 1, 0]
    ea.attn_pages_extend(pool, table, seqlens, _int([0, 0]), 16,
                         torch.empty(0, dtype=torch.int64, device="cuda"))
    assert ea.attn_last_device_error() == 0


def test_captured_steps():
    """Decode steps and their cut, captured once and replayed: the state moves on."""
    pages = Pages(64, 6, 20, 16)
    pool, table, seqlens = _state(pages, 6)
    new, keep = _int([3] * 6), _int([0] * 6)
    slots = torch.empty((6, 3), dtype=torch.int64, device="cuda")
    granted = torch.empty(6, dtype=torch.int32, device="cuda")

    def step():
        ea.attn_pages_extend(pool, table, seqlens, new, 16, slots, granted=granted)
        torch.sub(seqlens, 1, out=keep)          # one drafted token was wrong
        ea.attn_pages_trim(pool, table, seqlens, keep, 16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    _same(pages, pool, table, seqlens)
    for i in range(40):
        graph.replay()
        want = pages.extend([3] * 6)
        assert slots.tolist() == [row for row, _, _ in want] and granted.tolist() == [x for _, _, x in want]
        pages.trim([n - 1 for n in pages.len])
    _same(pages, pool, table, seqlens)


def test_on_another_stream():
    side = torch.cuda.Stream()
    pool = ea.page_pool(50, stream=side)
    with torch.cuda.stream(side):
        table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
        seqlens, new = _int([0, 0]), _int([20, 40])
    slots, pos, cu, granted = ea.pages_extend(pool, table, seqlens, new, 16, total=60, stream=side)
    ea.attn_pages_trim(pool, table, seqlens, new, 16, stream=side)
    side.synchronize()
    assert slots.tolist() == list(range(60 - 28)) [:20] + list(range(32, 72))
    assert pos.tolist() == list(range(20)) + list(range(40)) and seqlens.tolist() == [20, 40]


def test_serving_run():
    """Prompts into the cache and 70 decoded tokens with the bias, every table built on the
    GPU: each step's output equals attention over all keys so far, in 64 bits."""
    B, Hq, Hkv, d, page = 3, 4, 2, 64, 64
    lens = [50, 1, 130]
    g = torch.Generator().manual_seed(0)

    def randn(*s):
        return torch.randn(*s, generator=g).to(torch.bfloat16)
    buckets, first = ea.bias_buckets(32, 128)
    weights = torch.randn(32, Hq, generator=g)
    pool = ea.page_pool(12)
    table = torch.full((B, 5), -1, dtype=torch.int32, device="cuda")
    seqlens = torch.zeros(B, dtype=torch.int32, device="cuda")
    kp, vp = (torch.full((12, page, Hkv, d), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    # the prompts: packed
    q, k, v = randn(sum(lens), Hq, d), randn(sum(lens), Hkv, d), randn(sum(lens), Hkv, d)
    slots, pos, cu, granted = ea.pages_extend(pool, table, seqlens, _int(lens), page, total=sum(lens))
    ea.attn_cache_write(k.cuda(), v.cuda(), kp, vp, slots)
    o, lse = ea.forward_varlen_bias(q.cuda(), k.cuda(), v.cuda(), cu, cu, max(lens), max(lens), weights.cuda(),
                                    buckets, first, causal=True)
    ks, vs = list(k.split(lens)), list(v.split(lens))
    for b, (i0, n) in enumerate(zip([0, 50, 51], lens)):
        Problem(q[i0:i0 + n].transpose(0, 1), ks[b].transpose(0, 1), vs[b].transpose(0, 1), weights, buckets.cpu(),
                first, True).check_forward(o[i0:i0 + n].transpose(0, 1), lse[:, i0:i0 + n])
    # one token at a time
    for step in range(70):
        q, k, v = randn(B, Hq, 1, d), randn(B, Hkv, 1, d), randn(B, Hkv, 1, d)
        slots, pos, granted = ea.pages_extend(pool, table, seqlens, _int([1] * B), page, width=1)
        assert granted.tolist() == [1] * B and pos[:, 0].tolist() == [n + step for n in lens]
        ea.attn_cache_write(k.cuda(), v.cuda(), kp, vp, slots)
        o, lse = ea.decode_paged_bias(q.cuda(), kp, vp, table, seqlens, weights.cuda(), buckets, first)
        for b in range(B):
            ks[b] = torch.cat([ks[b], k[b].transpose(0, 1)])
            vs[b] = torch.cat([vs[b], v[b].transpose(0, 1)])
            if step % 23 == 0 or step == 69:
                Problem(q[b], ks[b].transpose(0, 1), vs[b].transpose(0, 1), weights, buckets.cpu(),
                        first).check_forward(o[b], lse[b])
    ea.pages_trim(pool, table, seqlens, _int([0] * B), page)
    assert sorted(pool[4:].tolist()) == list(range(12)) and pool[0] == 12
    assert ea.attn_last_device_error() == 0


def test_captured_decode_steps():
    """A whole decode step captured once (pages, the cache's write, attention with the bias) and
    replayed over 90 tokens, one sequence starting over on the way."""
    B, Hq, Hkv, d, page = 2, 4, 4, 128, 64
    g = torch.Generator().manual_seed(2)
    buckets, first = ea.bias_buckets(32, 128)
    weights = torch.randn(32, Hq, generator=g)
    pool = ea.page_pool(4)
    table = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
    seqlens = torch.zeros(B, dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros((4, page, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, k, v = (torch.zeros((B, h, 1, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    one, wg = _int([1] * B), weights.cuda()

    def step():
        slots, pos, granted = ea.pages_extend(pool, table, seqlens, one, page, width=1)
        ea.attn_cache_write(k, v, kp, vp, slots)
        return (pos, *ea.decode_paged_bias(q, kp, vp, table, seqlens, wg, buckets, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pos, o, lse = step()
    ks, vs = [[], []], [[], []]
    for n in range(90):
        if n == 40:      # sequence 1 is done, another begins in its place
            ea.attn_pages_trim(pool, table, seqlens, _int([1000, 0]), page)
            ks[1], vs[1] = [], []
        new = [torch.randn(B, h, 1, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]
        for dst, src in zip((q, k, v), new):
            dst.copy_(src)
        graph.replay()
        for b in range(B):
            ks[b].append(new[1][b])
            vs[b].append(new[2][b])
        assert pos[:, 0].tolist() == [len(x) - 1 for x in ks]
        if n % 13 == 0 or n == 89:
            for b in range(B):
                Problem(new[0][b], torch.cat(ks[b], 1), torch.cat(vs[b], 1), weights, buckets.cpu(),
                        first).check_forward(o[b], lse[b])
    assert ea.attn_last_device_error() == 0


def test_training_run():
    """Forward, backward and an update of the table, three times: each step's gradients are
    those of its table."""
    g = torch.Generator().manual_seed(1)
    q, k, v, dout = (torch.randn(1, 2, 200, 64, generator=g).to(torch.bfloat16) for _ in range(4))
    buckets, first = ea.bias_buckets(16, 64, True)
    table = torch.randn(16, 2, generator=g).cuda()
    for _ in range(3):
        o, lse = ea.forward_bias(q.cuda(), k.cuda(), v.cuda(), table, buckets, first, out_dtype=torch.float32)
        got = ea.backward_bias(q.cuda(), k.cuda(), v.cuda(), o, dout.cuda(), lse, table, buckets, first)
        ref = Problem(q[0], k[0], v[0], table.cpu(), buckets.cpu(), first)
        ref.check_forward(o[0], lse[0])
        grads, bounds = ref.gradients(o[0], dout[0], lse[0], 16)
        check_gradients([got[0][0], got[1][0], got[2][0], got[3]], grads, bounds)
        table = table - 0.5 * got[3]
