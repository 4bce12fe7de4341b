"""attn_decode_tree over an E4M3 cache whose V rows differ in size by many powers of two,
or leave a warp's keys without one that counts."""
import pytest
import torch

import exact_attention_14_gb300 as ea
from paged_ref import Cache, check_tree, tree64

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
