"""attn_decode_tree on the GPU against 64-bit attention over the cached values."""
import pytest
import torch

import exact_attention_14_gb300 as ea
from paged_ref import Cache, check_tree, random_trees, tree64

pytestmark = pytest.mark.gpu


def _q(B, Hq, T, d, seed=11, size=1.0):
    return (torch.randn(B, Hq, T, d, generator=torch.Generator().manual_seed(seed)) * size).to(torch.bfloat16)


def _run(q, cache, mask=None, q_lens=None, out=torch.float32, **kw):
    (kp, vp, table, sl), (kd, vd) = cache.on("cuda")
    o, lse = ea.decode_tree(q.cuda(), kp, vp, table, sl,
                            None if mask is None else ea.tree_mask_words(mask).cuda(),
                            None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32).cuda(),
                            kd, vd, out_dtype=out, **kw)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    return o.cpu(), lse.cpu()


SHAPES = [
    # lengths, Hq, Hkv, T, d, page
    ([1], 1, 1, 1, 64, 16), ([1, 2, 3], 2, 1, 1, 128, 64), ([64, 65, 63], 4, 2, 1, 128, 64),
    ([700, 1, 129], 8, 2, 1, 128, 16), ([7, 40, 300], 8, 2, 7, 96, 16), ([5], 4, 4, 5, 64, 32),
    ([70, 513], 8, 1, 16, 128, 48), ([200, 64], 16, 2, 33, 128, 64), ([300, 150], 16, 2, 64, 64, 16),
    ([257], 6, 2, 65, 80, 80), ([400], 4, 1, 130, 112, 128), ([260, 31], 24, 1, 3, 256, 32),
    ([600], 8, 2, 17, 192, 64), ([2000, 1, 90], 10, 5, 4, 32, 256),
]


@pytest.mark.parametrize("lengths,Hq,Hkv,T,d,page", SHAPES)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_matches_64_bits(lengths, Hq, Hkv, T, d, page, e4m3, tree):
    """Ragged drafts; pages that no table entry names and keys past a length are NaN."""
    B = len(lengths)
    q_lens = [min(T, n) - (min(T, n) // 2 if b % 2 else 0) for b, n in enumerate(lengths)]
    cache = Cache(lengths, Hkv, d, page, e4m3, seed=5, outliers=e4m3)
    q = _q(B, Hq, T, d)
    mask = random_trees(B, T, 3) if tree else None
    ref = tree64(q, cache, mask, q_lens)
    for out in (torch.float32, torch.bfloat16):
        o, lse = _run(q, cache, mask, q_lens, out)
        check_tree(o, lse, ref, e4m3, out)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("G,T", [(1, 1), (8, 1), (4, 16), (8, 64)])
def test_long_contexts_are_cut_and_merged(G, T, e4m3):
    """Every CTA takes a part of the one long sequence; its neighbours are short."""
    lengths = [9000, T, 70 + T, 3000]
    cache = Cache(lengths, 2, 128, 64, e4m3, seed=6)
    q = _q(4, 2 * G, T, 128)
    mask = random_trees(4, T, 4)
    o, lse = _run(q, cache, mask)
    check_tree(o, lse, tree64(q, cache, mask), e4m3, torch.float32)


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_that_attend_nothing(e4m3):
    """A mask that leaves a row empty, without and with a prefix; drafts of length 0."""
    T = 9
    cache = Cache([9, 20, 12, 0], 2, 64, 16, e4m3, seed=8)
    mask = random_trees(4, T, 5)
    mask[:, 2] = False                       # no prefix in sequence 0: row 2 sees nothing
    mask[:, 4, :] = False
    q_lens = [9, 9, 0, 0]
    q = _q(4, 6, T, 64)
    o, lse = _run(q, cache, mask, q_lens)
    assert (lse[0, :, 2] == -float("inf")).all() and (o[0, :, 4] == 0).all()
    assert torch.isfinite(lse[1, :, 2]).all()
    assert (lse[2:] == -float("inf")).all() and (o[2:] == 0).all()
    check_tree(o, lse, tree64(q, cache, mask, q_lens), e4m3, torch.float32)


@pytest.mark.parametrize("T,G", [(6, 1), (40, 4)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_unseen_drafts_may_hold_anything(T, G, what):
    """K and V of a drafted token that only some rows see: NaN or infinite, the
    other rows are as if it were not there, and the rows that see it are not finite."""
    lengths = [T + 50, T]
    cache = Cache(lengths, 2, 64, 16, seed=9)
    mask = random_trees(2, T, 6)
    bad = 3
    mask[:, bad + 1:, bad] = False
    mask[:, T - 1, bad] = True
    clean = Cache(lengths, 2, 64, 16, seed=9)
    q = _q(2, 2 * G, T, 64)
    for b, n in enumerate(lengths):
        slot = cache.slots[b][n - T + bad]
        cache.v_pages.view(-1, 2, 64)[slot, :, 5] = what
        if what != what:
            cache.k_pages.view(-1, 2, 64)[slot] = what
    o, lse = _run(q, cache, mask)
    ro, rl, size, eps = tree64(q, clean, mask)
    sees = mask[:, :, bad]
    rest = (~sees)[:, None, :].expand(2, 2 * G, T)
    rl = torch.where(rest, rl, torch.zeros_like(rl))
    check_tree(torch.where(rest[..., None], o, torch.zeros_like(o)), torch.where(rest, lse, torch.zeros_like(lse)),
               (ro * rest[..., None], rl, size, eps), False, torch.float32)
    seen = o[..., 5].masked_select(~rest)
    assert (seen != seen).all() if what != what else (seen == what).all()
    if what == what:     # the other columns of those rows are unharmed
        cols = torch.arange(64) != 5
        tol = (2 * (2.0 ** -8 + eps[..., None]) + 2.0 ** -18) * size * 1.02 + 1e-6
        assert ((o.double() - ro).abs() <= tol)[..., cols].all()


def test_unseen_drafts_may_hold_anything_e4m3():
    T, H, d = 12, 2, 128
    lengths = [T + 30, T]
    clean, cache = (Cache(lengths, H, d, 16, True, seed=10) for _ in range(2))
    mask = random_trees(2, T, 7)
    mask[:, 4:, 3] = False
    mask[:, 8:, 7] = False
    for b, n in enumerate(lengths):
        s3, s7 = cache.slots[b][n - T + 3], cache.slots[b][n - T + 7]
        cache.v_pages.view(-1, H, d)[s3, 0, 9] = 0x7F        # a NaN code
        cache.v_descale[s7 // 16, :, s7 % 16] = float("inf")
        cache.k_descale[s7 // 16, :, s7 % 16] = float("nan")
    q = _q(2, 4, T, d)
    o, lse = _run(q, cache, mask)
    ref = tree64(q, clean, mask)
    for t in range(T):
        if t in (3, 7):
            continue
        part = [x[:, :, t:t + 1] for x in ref]
        check_tree(o[:, :, t:t + 1], lse[:, :, t:t + 1], part, True, torch.float32)
    assert torch.isnan(o[:, :2, 3, 9]).all() and torch.isnan(o[:, :, 7]).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_dominant_key_and_many_small_ones(e4m3):
    """One key holds most of the weight and thousands of small ones the rest
    (P far below its largest value keeps its bits); V's rows differ in size."""
    n, d = 6000, 128
    g = torch.Generator().manual_seed(1)
    k = torch.randn(n, 1, d, generator=g) * 0.02
    q = torch.ones(1, 4, 1, d)
    k[0] = 1.0                                             # score 11.3, the others about 0
    v = torch.randn(n, 1, d, generator=g) + 1.0
    v[1:] *= torch.exp(torch.randn(n - 1, 1, 1, generator=g))
    cache = Cache([n], 1, d, 64, e4m3, k=[k.to(torch.bfloat16)], v=[v.to(torch.bfloat16)])
    q = (q + 0.1 * torch.randn(1, 4, 1, d, generator=g)).to(torch.bfloat16)
    o, lse = _run(q, cache)
    check_tree(o, lse, tree64(q, cache), e4m3, torch.float32)


def test_single_token_equals_decode_paged():
    """T = 1 over a bf16 cache computes what attn_decode_paged computes."""
    cache = Cache([900, 33, 1], 2, 128, 64, seed=12, max_blocks=16)
    q = _q(3, 8, 1, 128)
    (kp, vp, table, sl), _ = cache.on("cuda")
    o, lse = _run(q, cache)
    o2, l2 = ea.decode_paged(q.cuda(), kp, vp, table, sl, out_dtype=torch.float32)
    ref = tree64(q, cache)
    check_tree(o2.cpu(), l2.cpu(), ref, False, torch.float32)
    check_tree(o, lse, ref, False, torch.float32)


def test_bad_lengths_are_reported_and_leave_the_rest():
    cache = Cache([50, 60, 70, 80], 2, 64, 16, seed=13)
    q = _q(4, 4, 8, 64)
    ref = tree64(q, cache)
    (kp, vp, table, sl), _ = cache.on("cuda")
    lens = torch.tensor([8, 9, 8, -1], dtype=torch.int32).cuda()      # more than T, and negative
    sl[0] = table.shape[1] * 16 + 1                                    # past the table
    o, lse = ea.decode_tree(q.cuda(), kp, vp, table, sl, None, lens, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    for b in (0, 1, 3):
        assert (o[b] == 0).all() and (lse[b] == -float("inf")).all()
    check_tree(o[2:3].cpu(), lse[2:3].cpu(), [x[2:3] for x in ref], False, torch.float32)


@pytest.mark.parametrize("T", [1, 20])
def test_same_bits_again_on_a_stream_and_in_a_graph(T):
    cache = Cache([5000, 700, 64], 2, 128, 64, True, seed=14)
    q = _q(3, 8, T, 128)
    o, lse = _run(q, cache)
    (kp, vp, table, sl), (kd, vd) = cache.on("cuda")
    s = torch.cuda.Stream()
    qc = q.cuda()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, l2 = ea.decode_tree(qc, kp, vp, table, sl, None, None, kd, vd, out_dtype=torch.float32)
    s.synchronize()
    assert torch.equal(o2.cpu(), o) and torch.equal(l2.cpu(), lse)
    o3, l3 = ea.decode_tree(qc, kp, vp, table, sl, None, None, kd, vd, out_dtype=torch.float32, stream=s)
    s.synchronize()
    assert torch.equal(o3.cpu(), o)
    ws = torch.empty(ea.attn_decode_tree_workspace_size(3, 8, 2, T, table.shape[1], 64, 128, True),
                     dtype=torch.uint8, device="cuda")
    og, lg = torch.zeros_like(o2), torch.zeros_like(l2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ea.attn_decode_tree(qc, kp, vp, table, sl, og, lg, None, None, kd, vd, workspace=ws)
    ws.fill_(255)                                             # its contents do not matter
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(og.cpu(), o) and torch.equal(lg.cpu(), lse)
    sl -= 13                                                  # lengths are read when it runs
    g.replay()
    torch.cuda.synchronize()
    cache.seqlens -= 13
    assert torch.equal(og.cpu(), _run(q, cache)[0])
    assert ea.attn_last_device_error() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_decode_step_and_a_chunk(e4m3):
    """Positions, cache and attention as a server runs them: a prompt is written
    to the cache, drafted tokens are rotated, written and attended over it; and
    the same rows come out of the cache read back through attn_fwd_varlen."""
    B, Hq, Hkv, T, d, page = 2, 8, 2, 6, 128, 16
    prompts = [77, 40]
    g = torch.Generator().manual_seed(3)
    f, mag = ea.rope_frequencies(d, scaling="linear", factor=2.0)
    width = 8
    kind = torch.uint8 if e4m3 else torch.bfloat16
    kp = torch.zeros(B * width, page, Hkv, d, dtype=kind, device="cuda")
    vp = torch.zeros_like(kp)
    kd = torch.ones(B * width, Hkv, page, device="cuda") if e4m3 else None
    vd = kd.clone() if e4m3 else None
    table = torch.randperm(B * width, generator=g).reshape(B, width).to(torch.int32).cuda()

    def slots(b, pos):
        return table[b].long()[pos // page] * page + pos % page

    def new(*shape):
        return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()
    for b, n in enumerate(prompts):
        pos = torch.arange(n, device="cuda")
        k, _ = ea.rope(new(n, Hkv, d), None, pos.int(), f, magnitude=mag)
        ea.attn_cache_write(k, new(n, Hkv, d), kp, vp, slots(b, pos), kd, vd)
    # drafted tokens, token-major as a projection leaves them
    pos = torch.tensor(prompts)[:, None].cuda() + torch.arange(T, device="cuda")
    qkv = new(B, T, Hq + 2 * Hkv, d)
    q, k = ea.rope(qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hkv].transpose(1, 2), pos.int(), f,
                   magnitude=mag)
    at = torch.stack([slots(b, pos[b]) for b in range(B)])
    ea.attn_cache_write(k, qkv[:, :, Hq + Hkv:].transpose(1, 2), kp, vp, at, kd, vd)
    sl = torch.tensor(prompts, dtype=torch.int32).cuda() + T
    o, lse = ea.decode_tree(q, kp, vp, table, sl, None, None, kd, vd)
    # the same through the cache read back
    cu_k = torch.tensor([0] + [n + T for n in prompts]).cumsum(0).to(torch.int32).cuda()
    cu_q = torch.arange(0, B * T + 1, T, dtype=torch.int32, device="cuda")
    kk, vv = ea.cache_read(kp, vp, table, cu_k, int(cu_k[-1]), kd, vd)
    o2, l2 = ea.forward_varlen(q.transpose(1, 2).reshape(B * T, Hq, d), kk, vv, cu_q, cu_k, T,
                               max(prompts) + T, causal=True)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    o2 = o2.reshape(B, T, Hq, d).transpose(1, 2)
    l2 = l2.reshape(Hq, B, T).transpose(0, 1)
    # both round P to bf16 (or finer) and O to bf16; the read-back rounds E4M3 values to bf16:
    # keys off by 2^-8 move a score by at most 2^-8 * scale * sum |q||k|
    eps = 2.0 ** -8 * d ** -0.5 * (q.float().abs().sum(-1) * kk.float().abs().max()).max().item() if e4m3 else 0.0
    size = vv.float().abs().max().item()
    assert (o.float() - o2.float()).abs().max() <= (6 * 2.0 ** -8 + 2 * eps) * size
    assert (lse - l2).abs().max() <= eps + 2.0 ** -12
