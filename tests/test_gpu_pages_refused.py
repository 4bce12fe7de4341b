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


def _packed(new, total, page=16, blocks=40, max_blocks=8, held=None):
    """One packed extend: (slots with a guard behind them, positions, cu_seqlens, granted,
    lengths, free pages, the tables)."""
    B = len(new)
    pool = ea.page_pool(blocks)
    table = torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda")
    seqlens = torch.zeros(B, dtype=torch.int32, device="cuda")
    if held is not None:
        ea.pages_extend(pool, table, seqlens, _int(held), page, total=sum(held))
    slots = torch.full((total + 4,), 77, dtype=torch.int64, device="cuda")
    pos = torch.full((total + 4,), 77, dtype=torch.int32, device="cuda")
    cu, granted = torch.empty(B + 1, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    ea.attn_pages_extend(pool, table, seqlens, _int(new), page, slots[:total], pos[:total], cu, granted)
    assert (slots[total:] == 77).all() and (pos[total:] == 77).all()
    return slots[:total].tolist(), pos[:total].tolist(), cu.tolist(), granted.tolist(), seqlens.tolist(), pool, table


def test_packed_rows_for_fewer_tokens():
    """From the first request whose tokens end past the rows on, new tokens count as none: no
    length holds a token without a slot, and no page is taken for one."""
    held = [5, 0, 30, 16, 1]
    slots, pos, cu, granted, lens, pool, table = _packed([4, 0, 20, 1, 0], 10, held=held)
    _reported()
    # (held: page 0 for request 0, 1 and 2 for request 2, 3 for request 3, 4 for request 4)
    assert slots == [5, 6, 7, 8] + [-1] * 6 and pos == [5, 6, 7, 8] + [0] * 6
    assert cu == [0, 4, 4, 4, 4, 4] and granted == [4, 0, 0, 0, 0]
    assert lens == [9, 0, 30, 16, 1] and pool[0] == 35 and (table[3, 1:] == -1).all()
    # the same with a row more than all of them need, and with as many
    for total in (26, 25):
        slots, pos, cu, granted, lens, pool, _ = _packed([4, 0, 20, 1, 0], total, held=held)
        assert ea.attn_last_device_error() == 0
        assert cu == [0, 4, 4, 24, 25, 25] and granted == [4, 0, 20, 1, 0] and lens == [9, 0, 50, 17, 1]
        assert (-1 in slots) == (total == 26) and pool[0] == 35 - 3
    # one row short: the last request that has any gets none
    slots, pos, cu, granted, lens, pool, _ = _packed([4, 0, 20, 1, 0], 24, held=held)
    _reported()
    assert cu == [0, 4, 4, 24, 24, 24] and granted == [4, 0, 20, 0, 0] and lens == [9, 0, 50, 16, 1]
    assert -1 not in slots and pool[0] == 35 - 2
    # no rows at all
    slots, pos, cu, granted, lens, pool, _ = _packed([4, 0, 20, 1, 0], 0, held=held)
    _reported()
    assert cu == [0] * 6 and granted == [0] * 5 and lens == held and pool[0] == 35


def test_packed_rows_and_pages_that_both_run_out():
    """Rows end at request 3, pages at request 1: what is served fits both."""
    slots, pos, cu, granted, lens, pool, _ = _packed([16, 40, 10, 50], 70, blocks=3)
    _reported()
    assert cu == [0, 16, 56, 66, 66] and granted == [16, 0, 0, 0] and lens == [16, 0, 0, 0]
    assert slots == list(range(16)) + [-1] * 54 and pool[0] == 2


@pytest.mark.parametrize("B", [257, 2000])
def test_packed_rows_of_many_requests(B):
    """Several requests a thread: the border lies inside a thread's share, and past it."""
    new = [(7 * b) % 5 for b in range(B)]
    ends = torch.tensor(new).cumsum(0).tolist()
    for at in (0, 1, B // 3, B - 2):
        total = ends[at] + 1        # (below the next request with 2 or more tokens' end)
        fits = [e <= total for e in ends]
        want = [n if ok else 0 for n, ok in zip(new, fits)]
        slots, pos, cu, granted, lens, pool, _ = _packed(want, total, blocks=2 * B)
        assert ea.attn_last_device_error() == 0
        got = _packed(new, total, blocks=2 * B)
        _reported()
        assert got[:5] == (slots, pos, cu, granted, lens) and torch.equal(got[5], pool)
        assert granted == want and lens == want and cu[-1] == sum(want)


def test_packed_sums_past_31_bits():
    """Requests of 2^24 tokens, one page each: the sums pass 2^31, lengths and pages do not
    drift apart."""
    page, B = 1 << 24, 200
    slots, pos, cu, granted, lens, pool, table = _packed([page] * B, 50, page=page, blocks=B, max_blocks=1)
    _reported()
    assert lens == [0] * B and granted == [0] * B and cu == [0] * (B + 1)
    assert pool[0] == B and (table == -1).all() and slots == [-1] * 50
