"""attn_decode_tree at the borders of its variants, with pages that are missing, on
other streams, and many times over."""
import pytest
import torch

import exact_attention_14_gb300 as ea
from paged_ref import Cache, check_tree, quantize, random_trees, rope64, tree64

pytestmark = pytest.mark.gpu


def _q(B, Hq, T, d, seed=21):
    return torch.randn(B, Hq, T, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _args(q, cache, mask=None, q_lens=None):
    (kp, vp, table, sl), (kd, vd) = cache.on("cuda")
    return [q.cuda(), kp, vp, table, sl, None if mask is None else ea.tree_mask_words(mask).cuda(),
            None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32).cuda(), kd, vd]


def _run(*a, **kw):
    o, lse = ea.decode_tree(*_args(*a), out_dtype=torch.float32, **kw)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    return o.cpu(), lse.cpu()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,T", [(8, 1), (3, 3), (4, 4), (1, 17), (2, 9), (16, 8), (3, 43), (4, 64), (257, 1), (5, 77)])
def test_row_counts_around_the_tiles(G, T, e4m3):
    """G * T = 8, 9, 16, 17, 18, 128, 129, 256, 257, 385 query rows a head of the cache."""
    lengths = [T + 300, T, T + 1]
    cache = Cache(lengths, 1, 64, 32, e4m3, seed=22)
    q = _q(3, G, T, 64)
    mask = random_trees(3, T, 8)
    q_lens = [T, T, (T + 1) // 2]
    o, lse = _run(q, cache, mask, q_lens)
    check_tree(o, lse, tree64(q, cache, mask, q_lens), e4m3, torch.float32)


@pytest.mark.parametrize("T", [1, 12])
def test_many_sequences(T):
    """More sequences than lanes of a warp, empty ones and ones without drafts among them."""
    g = torch.Generator().manual_seed(1)
    B = 150
    lengths = [int(x) for x in torch.randint(0, 90, (B,), generator=g)]
    q_lens = [0 if b % 11 == 5 else min(T, n) for b, n in enumerate(lengths)]
    cache = Cache(lengths, 1, 64, 16, T > 1, seed=23)
    q = _q(B, 2, T, 64)
    o, lse = _run(q, cache, None, q_lens)
    check_tree(o, lse, tree64(q, cache, None, q_lens), T > 1, torch.float32)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_thousand_drafts(e4m3):
    """The most tokens a mask can hold are 1024; here 1000 as a chunk of a prompt, and 999 with
    a mask of 16 words a row."""
    cache = Cache([1000 + 130], 1, 64, 16, e4m3, seed=24)
    q = _q(1, 1, 1000, 64)
    o, lse = _run(q, cache)
    check_tree(o, lse, tree64(q, cache), e4m3, torch.float32)
    mask = random_trees(1, 1000, 9)
    o, lse = _run(q, cache, mask, [999])
    check_tree(o, lse, tree64(q, cache, mask, [999]), e4m3, torch.float32)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [2, 40])
def test_missing_pages_read_as_zeros(T, e4m3):
    """Table entries that name no page, while page 0 and every other one hold NaN where no
    sequence lies."""
    lengths, page = [T + 200, T + 64], 16
    zeroed = [(0, 3), (0, 4), (1, 0)]                          # (sequence, block of its table)
    k, v = ([torch.randn(n, 2, 64, generator=torch.Generator().manual_seed(25 + i)).to(torch.bfloat16)
             for n in lengths] for i in (0, 1))
    for b, blk in zeroed:
        k[b][blk * page:(blk + 1) * page] = 0
        v[b][blk * page:(blk + 1) * page] = 0
    cache = Cache(lengths, 2, 64, page, e4m3, seed=26, k=k, v=v)
    q = _q(2, 4, T, 64)
    ref = tree64(q, cache)
    for i, (b, blk) in enumerate(zeroed):
        old = int(cache.table[b, blk])
        for x, fill in ((cache.k_pages, 0x7F if e4m3 else float("nan")), (cache.k_descale, float("nan"))):
            if x is not None:
                x[old] = fill
        cache.table[b, blk] = (-1, 2 ** 29, -2 ** 31)[i]
    # page 0 not in use by any sequence: its rows change places with a spare page's
    spare = cache.k_pages.shape[0]
    for name in ("k_pages", "v_pages", "k_descale", "v_descale"):
        x = getattr(cache, name)
        if x is not None:
            x = torch.cat([x, x[:1]])
            x[0] = 0x7F if x.dtype == torch.uint8 else float("nan")
            setattr(cache, name, x)
    cache.table[cache.table == 0] = spare
    o, lse = _run(q, cache)
    check_tree(o, lse, ref, e4m3, torch.float32)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,T", [(1, 2), (4, 8)])
def test_queries_that_are_not_finite(G, T, e4m3):
    """Rows of Q with a NaN or an infinity give NaN; their neighbours are as ever."""
    cache = Cache([T + 100], 2, 64, 16, e4m3, seed=27)
    q = _q(1, 2 * G, T, 64)
    ref = tree64(q, cache)
    q[0, 0, 0, 7] = float("nan")
    q[0, 2 * G - 1, T - 1, 0] = float("inf")
    o, lse = _run(q, cache)
    for h, t in ((0, 0), (2 * G - 1, T - 1)):
        assert torch.isnan(o[0, h, t]).all() and torch.isnan(lse[0, h, t])
        o[0, h, t], lse[0, h, t] = ref[0][0, h, t].float(), ref[1][0, h, t].float()
    check_tree(o, lse, ref, e4m3, torch.float32)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,T", [(4, 1), (4, 16), (4, 64)])
def test_the_same_bits_a_thousand_times(G, T, e4m3):
    """Launches behind one another, each CTA's work cut in the middle of sequences: no wait
    runs out and no bit changes."""
    lengths = [T + 3000, T, T + 700, 9000]
    cache = Cache(lengths, 4, 128, 64, e4m3, seed=28)
    a = _args(_q(4, 4 * G, T, 128), cache, random_trees(4, T, 10))
    first = ea.decode_tree(*a)
    graph = torch.cuda.CUDAGraph()
    outs = []
    with torch.cuda.graph(graph):
        for _ in range(50):
            outs.append(ea.decode_tree(*a))
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    for o, lse in outs:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_outputs_of_a_call_on_another_stream():
    """What a call on stream= allocates is not memory that queued work of the current stream
    still writes."""
    B, H, N, d = 2, 4, 64, 64
    cache = Cache([N, N], 2, d, 16, seed=29)
    a = _args(_q(B, H, 4, d), cache)
    q = _q(B, H, N, d).cuda()
    f, _ = ea.rope_frequencies(d)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, N, 2 * N], dtype=torch.int32, device="cuda")
    calls = (lambda **kw: ea.rope(q, q, pos, f, **kw),
             lambda **kw: ea.decode_tree(*a, **kw),
             lambda **kw: ea.cache_read(a[1], a[2], a[3], cu, 2 * N, **kw))
    for call in calls:
        want = [x.clone() for x in call()]
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        for stream in (s, s.cuda_stream):
            old = [torch.empty_like(x) for x in want for _ in range(4)]
            torch.cuda._sleep(20_000_000)                       # about ten milliseconds of the current stream
            for x in old:
                x.fill_(7)
            del old, x
            got = call(stream=stream)
            torch.cuda.synchronize()
            for x, y in zip(got, want):
                assert torch.equal(x, y)
            del got, x, y
    assert ea.attn_last_device_error() == 0


def test_two_graphs_with_their_own_workspaces():
    """Two captured calls of different shapes replayed side by side on two streams."""
    runs = []
    for i, (T, e4m3) in enumerate(((1, True), (24, False))):
        cache = Cache([4000, 900, 33 + T], 2, 128, 64, e4m3, seed=30 + i)
        a = _args(_q(3, 8, T, 128), cache)
        want = ea.decode_tree(*a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = ea.decode_tree(*a)
        runs.append((graph, torch.cuda.Stream(), got, want, a))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s, *_ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    for _, _, got, want, _ in runs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("e4m3", [False, True])
def test_positions_cache_and_gradients_of_one_buffer(e4m3):
    """q, k and v as slices of one projection, its gradient's slices rotated back in place,
    and the keys written as the write's definition says."""
    B, Hq, Hkv, N, d, page = 2, 4, 2, 33, 64, 16
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=torch.Generator().manual_seed(31)).to(torch.bfloat16)
    y = x.cuda()
    f, mag = ea.rope_frequencies(d, 500000.0)
    pos = (torch.arange(N) * 7 + 100000).to(torch.int32)
    q, k, v = (z.transpose(1, 2) for z in y.split([Hq, Hkv, Hkv], 2))
    ea.attn_rope(q, k, q, k, pos.cuda(), f, magnitude=mag)
    ref, size = rope64(x[:, :, :Hq + Hkv].transpose(1, 2), pos, f.cpu())
    got = y[:, :, :Hq + Hkv].transpose(1, 2).double().cpu()
    assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * size).all()
    assert torch.equal(y[:, :, Hq + Hkv:].cpu(), x[:, :, Hq + Hkv:])
    kind = torch.uint8 if e4m3 else torch.bfloat16
    kp = torch.zeros(6, page, Hkv, d, dtype=kind, device="cuda")
    vp = torch.zeros_like(kp)
    kd, vd = (torch.zeros(6, Hkv, page, device="cuda") if e4m3 else None for _ in range(2))
    slots = torch.arange(B * N).view(B, N)
    slots[1, 5] = -1
    ea.attn_cache_write(k, v, kp, vp, slots.cuda(), kd, vd)
    rows = k.transpose(1, 2).reshape(B * N, Hkv, d).cpu()
    keep = slots.flatten() >= 0
    flat = kp.view(-1, Hkv, d)[:B * N].cpu()
    if e4m3:
        codes, ds = quantize(rows)
        assert torch.equal(flat[keep], codes[keep])
        assert torch.equal(kd.transpose(1, 2).reshape(-1, Hkv)[:B * N].cpu()[keep], ds[keep])
    else:
        assert torch.equal(flat[keep], rows[keep])
    assert (flat[~keep] == 0).all()
    # the same places hold gradients: rotated back, they are the transposed rotation's
    g = torch.randn(B, N, Hq + 2 * Hkv, d, generator=torch.Generator().manual_seed(32)).cuda()
    want, size = rope64(g[:, :, :Hq + Hkv].transpose(1, 2).cpu(), pos, f.cpu(), inverse=True)
    dq, dk = g[:, :, :Hq].transpose(1, 2), g[:, :, Hq:Hq + Hkv].transpose(1, 2)
    ea.attn_rope(dq, dk, dq, dk, pos.cuda(), f, inverse=True, magnitude=mag)
    got = g[:, :, :Hq + Hkv].transpose(1, 2).double().cpu()
    assert ((got - want).abs() <= 2.0 ** -20 * size).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,T", [(1, 9), (4, 70)])
def test_mask_bits_past_the_drafts_count_for_nothing(G, T, e4m3):
    """Words of ones: every drafted token sees all n_b of its sequence, and no more."""
    lengths, q_lens = [T + 40, T - 3, T], [T, T - 3, 5]
    cache = Cache(lengths, 2, 64, 16, e4m3, seed=33)
    q = _q(3, 2 * G, T, 64)
    a = _args(q, cache, torch.ones(3, T, T, dtype=torch.bool), q_lens)
    a[5].fill_(-1)
    o, lse = ea.decode_tree(*a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    ref = tree64(q, cache, torch.ones(3, T, T, dtype=torch.bool), q_lens)
    check_tree(o.cpu(), lse.cpu(), ref, e4m3, torch.float32)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,T", [(2, 3), (2, 24), (4, 60)])
def test_bad_lengths_leave_the_other_sequences(G, T, e4m3):
    """Lengths past the table, drafts past T or past the keys, negative ones: zeros and an error,
    in each kernel, with the sequences between them as ever."""
    lengths = [T + 50, T + 9, 2 * T, T + 300, T + 1]
    cache = Cache(lengths, 2, 128, 16, e4m3, seed=34)
    q = _q(5, 2 * G, T, 128)
    ref = tree64(q, cache)
    a = _args(q, cache, None, [T] * 5)
    a[4][0] = a[3].shape[1] * 16 + 1
    a[6][2] = T + 1
    a[4][4] = -3
    o, lse = ea.decode_tree(*a, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    for b in (0, 2, 4):
        assert (o[b] == 0).all() and (lse[b] == -float("inf")).all()
    for b in (1, 3):
        check_tree(o[b:b + 1].cpu(), lse[b:b + 1].cpu(), [x[b:b + 1] for x in ref], e4m3, torch.float32)
    a[4].copy_(torch.tensor(lengths, dtype=torch.int32))
    a[6].fill_(T)
    o, lse = ea.decode_tree(*a, out_dtype=torch.float32)           # and the next call is whole again
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    check_tree(o.cpu(), lse.cpu(), ref, e4m3, torch.float32)
