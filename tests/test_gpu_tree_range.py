"""attn_decode_tree over an E4M3 cache whose V rows differ in size by many powers of two,
or leave a warp's keys without one that counts."""
import pytest
import torch

import exact_attention_14_gb300 as ea
from paged_ref import Cache, check_tree, random_trees, tree64

pytestmark = pytest.mark.gpu

INF = float("inf")


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _args(q, cache, mask=None):
    (kp, vp, table, sl), (kd, vd) = cache.on("cuda")
    return [q.cuda(), kp, vp, table, sl, None if mask is None else ea.tree_mask_words(mask).cuda(), None, kd, vd]


def _run(q, cache, mask=None):
    o, lse = ea.decode_tree(*_args(q, cache, mask), out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    return o.cpu(), lse.cpu()


def _spoil(cache, b, key, how):
    """Makes the V row of a key hold nothing that a row may use."""
    slot, page = int(cache.slots[b][key]), cache.page
    if how == "nan code":
        cache.v_pages.view(-1, *cache.v_pages.shape[2:])[slot] = 0x7F
    elif how == "no page":
        assert key % page == 0 and key == cache.lengths[b] - 1
        cache.table[b, key // page] = 2 ** 30
    else:
        cache.v_descale[slot // page, :, slot % page] = {"inf descale": INF, "zero descale": 0.0}[how]


SPOILED = ["nan code", "inf descale", "zero descale", "no page"]


@pytest.mark.parametrize("how", SPOILED)
@pytest.mark.parametrize("d,Hq", [(64, 1), (128, 8), (128, 12), (256, 2), (128, 40)])
def test_the_lone_key_of_a_slice_is_unseen(d, Hq, how):
    """33 keys, the last one a drafted token that not even its own row sees: the warp that holds
    it has no key at all, and the other 32 are the answer."""
    clean, cache = (Cache([33, 97], 1, d, 16, True, seed=41) for _ in range(2))
    for b, n in enumerate(cache.lengths):
        _spoil(cache, b, n - 1, how)
    q = _randn(2, Hq, 1, d, seed=42).to(torch.bfloat16)
    mask = torch.zeros(2, 1, 1, dtype=torch.bool)
    o, lse = _run(q, cache, mask)
    check_tree(o, lse, tree64(q, clean, mask), True, torch.float32)


@pytest.mark.parametrize("how", SPOILED)
@pytest.mark.parametrize("d,G", [(256, 1), (256, 3), (128, 1)])
def test_a_chain_whose_last_slice_most_rows_do_not_see(d, G, how):
    """33 drafted tokens without a prefix, the last one's V row spoiled: rows 0..31 do not see it."""
    T = 33
    clean, cache = (Cache([T], 1, d, 16, True, seed=43) for _ in range(2))
    _spoil(cache, 0, T - 1, how)
    q = _randn(1, G, T, d, seed=44).to(torch.bfloat16)
    o, lse = _run(q, cache)
    ref = tree64(q, clean)
    check_tree(o[:, :, :T - 1], lse[:, :, :T - 1], [x[:, :, :T - 1] for x in ref], True, torch.float32)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,G,T", [(128, 8, 1), (64, 4, 3), (256, 2, 1), (256, 4, 5), (128, 1, 20), (128, 4, 64)])
def test_values_up_to_the_largest_bf16(d, G, T, out):
    """V rows of 1.6e38..3.2e38, written by attn_cache_write; every row's average of them is finite."""
    lengths, H, page = [2100, T + 40, T], 2, 64
    v = [((1 + torch.rand(n, H, d, generator=torch.Generator().manual_seed(45 + i))) * 1.6e38).to(torch.bfloat16)
         for i, n in enumerate(lengths)]
    cache = Cache(lengths, H, d, page, True, seed=46, v=v)
    q = _randn(3, H * G, T, d, seed=47).to(torch.bfloat16)
    a = _args(q, cache)
    for pages, descale in ((a[1], a[7]), (a[2], a[8])):
        pages.fill_(0x7F)
        descale.fill_(float("nan"))
    ea.attn_cache_write(torch.cat(cache.k).cuda(), torch.cat(v).cuda(), a[1], a[2], torch.cat(cache.slots).cuda(),
                        a[7], a[8])
    o, lse = ea.decode_tree(*a, out_dtype=out)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    assert torch.isfinite(o).all()
    check_tree(o, lse, tree64(q, cache), True, out)


ROWS = [(128, 1, 6), (64, 2, 8), (256, 1, 12), (256, 4, 6), (128, 1, 20), (64, 4, 20), (128, 4, 60)]


@pytest.mark.parametrize("size", [1e-30, 1e6, 1e30, 3e38])
@pytest.mark.parametrize("prefix", [0, 50, 700])
@pytest.mark.parametrize("d,G,T", ROWS)
def test_unseen_drafts_of_any_finite_size(d, G, T, prefix, size):
    """A drafted token whose V row is far larger (or smaller) than the others': rows that do not see
    it keep every bit, and so do rows that do."""
    lengths = [T + prefix, T + prefix // 2]
    v = [_randn(n, 1, d, seed=48 + i) for i, n in enumerate(lengths)]
    for x in v:
        x[-T + 3] *= size / x[-T + 3].abs().max()
    cache = Cache(lengths, 1, d, 16, True, seed=49, v=[x.to(torch.bfloat16) for x in v])
    mask = random_trees(2, T, 50)
    mask[:, 4:, 3] = False
    mask[:, T - 1, 3] = True
    q = _randn(2, G, T, d, seed=51).to(torch.bfloat16)
    o, lse = _run(q, cache, mask)
    check_tree(o, lse, tree64(q, cache, mask), True, torch.float32)


def _descale_floor(q, cache, mask, unit, one):
    """What a row's V rows may be off by, apart from their own roundings, where they are held in
    steps of `unit` times the largest descale that the row sees: sum_j (|code_j| + one) * unit * that."""
    B, Hq, T, d = q.shape
    out = torch.zeros(B, Hq, T, d, dtype=torch.float64)
    for b in range(B):
        L = cache.lengths[b]
        codes = cache.v_pages.view(-1, *cache.v_pages.shape[2:])[cache.slots[b]].view(torch.float8_e4m3fn).double().abs()
        ds = cache.v_descale[cache.slots[b] // cache.page, :, cache.slots[b] % cache.page].double()
        see = torch.ones(T, L, dtype=torch.bool)
        see[:, L - T:] = torch.tril(torch.ones(T, T, dtype=torch.bool)) if mask is None else mask[b]
        for h in range(Hq):
            kv = h // (Hq // ds.shape[1])
            for t in range(T):
                js = see[t].nonzero().squeeze(1)
                if js.numel():
                    out[b, h, t] = unit * ds[js, kv].max() * (codes[js, kv] + one).sum(0)
    return out


@pytest.mark.parametrize("d,G,T", ROWS)
def test_drafts_of_all_sizes_without_a_prefix(d, G, T):
    """V rows from 1e-12 to 1e12, seen by some rows and not by others."""
    v = _randn(T, 1, d, seed=52) * 10.0 ** (24 * torch.rand(T, 1, 1, generator=torch.Generator().manual_seed(53)) - 12)
    cache = Cache([T], 1, d, 16, True, seed=54, v=[v.to(torch.bfloat16)])
    mask = random_trees(1, T, 55)
    q = _randn(1, G, T, d, seed=56).to(torch.bfloat16)
    o, lse = _run(q, cache, mask)
    ro, rl, size, eps = tree64(q, cache, mask)
    if T * G <= 16 or d > 128:
        # weights times descales are held in fp16 times 2^15 over a power of two that is at most
        # twice the row's largest descale: steps of 2^-24, half of one, 2^-39 of it; a weight
        # relative to the largest one, over a sum of at least 1
        size = size + _descale_floor(q, cache, mask, 2.0 ** -39, 0) / (3 * 2.0 ** -11)
    check_tree(o, lse, (ro, rl, size, eps), True, torch.float32)


@pytest.mark.parametrize("big", [1e3, 1e6, 1e8])
@pytest.mark.parametrize("d,G,T", [(128, 8, 1), (64, 2, 3), (256, 1, 2), (256, 2, 20), (128, 1, 20), (128, 4, 40)])
def test_a_large_value_of_almost_no_weight(d, G, T, big):
    """A key of the context with a large V row and next to no weight: the others keep the bits that
    the documentation says."""
    n = 400
    k, v = _randn(n, 1, d, seed=57) * 0.5, _randn(n, 1, d, seed=58)
    q = _randn(1, G, T, d, seed=59) * 0.3 + 1.0
    k[5] = -30.0 / d ** 0.5                                          # q . k / sqrt(d) about -30
    v[5] *= big
    cache = Cache([n], 1, d, 16, True, k=[k.to(torch.bfloat16)], v=[v.to(torch.bfloat16)])
    q = q.to(torch.bfloat16)
    o, lse = _run(q, cache)
    ro, rl, size, eps = tree64(q, cache)
    if T * G <= 16 or d > 128:
        size = size + _descale_floor(q, cache, None, 2.0 ** -39, 0) / (3 * 2.0 ** -11)
    else:
        # code * fp16(2^7 descale / F), F at most twice the largest descale: the factor and the product
        # are in steps of 2^-24, half of one over 2^7 is 2^-31 of that descale
        size = size + _descale_floor(q, cache, None, 2.0 ** -31, 1) / (3 * 2.0 ** -11)
    check_tree(o, lse, (ro, rl, size, eps), True, torch.float32)
