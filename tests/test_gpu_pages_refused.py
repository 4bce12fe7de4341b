"""The paged cache's tables on the GPU: calls that they cannot serve, or serve in part,
leave a pool, lengths and tables that the calls after them can use."""
import pytest
import torch

import exact_attention_14_gb300 as ea

pytestmark = pytest.mark.gpu


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _reported():
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [-1, 200, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("B,max_blocks", [(3, 8), (300, 20)])     # one block of threads, and several
def test_trim_of_what_is_no_page(B, max_blocks, bad):
    """An entry to give back that names no page: reported, and the whole call without effect."""
    page, blocks, at = 16, 200, B // 2
    pool = ea.page_pool(blocks)
    table = torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda")
    seqlens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = [0] * B
    new[0], new[at], new[-1] = 40, 60, 17
    ea.pages_extend(pool, table, seqlens, _int(new), page, total=sum(new))
    good = table[at, 2].item()
    table[at, 2] = bad
    before = pool[:4 + blocks].clone(), table.clone(), seqlens.clone()
    ea.attn_pages_trim(pool, table, seqlens, torch.zeros_like(seqlens), page)
    _reported()
    free = before[0][0].item()
    assert torch.equal(pool[:4 + free], before[0][:4 + free])
    assert torch.equal(table, before[1]) and torch.equal(seqlens, before[2])
    # a cut that keeps the entry's page gives back the others'
    keep = [0] * B
    keep[at] = 33                     # pages 0, 1 and 2 of the request stay, page 3 goes
    last = table[at, 3].item()
    ea.attn_pages_trim(pool, table, seqlens, _int(keep), page)
    assert ea.attn_last_device_error() == 0
    assert seqlens.tolist() == keep and pool[:4].tolist() == [blocks - 3, 0, 0, 0]
    assert last in pool[4:1 + blocks].tolist()
    # the entry put right, everything comes back and every page goes out once
    table[at, 2] = good
    ea.attn_pages_trim(pool, table, seqlens, torch.zeros_like(seqlens), page)
    assert pool[0] == blocks and sorted(pool[4:].tolist()) == list(range(blocks))
    slots, _, granted = ea.pages_extend(pool, table, seqlens, _int(new), page, width=60)
    assert granted.tolist() == new and (slots >= 0).sum() == sum(new)
    assert ea.attn_last_device_error() == 0
