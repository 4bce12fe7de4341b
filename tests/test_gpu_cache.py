"""Writing and reading the paged cache on the GPU: codes and descales bit for
bit against the fp32 formula, values against 64 bits."""
import pytest
import torch

import exact_attention_14_gb300 as ea
from paged_ref import HALF, Cache, quantize

pytestmark = pytest.mark.gpu


def _rows(B, H, N, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, N, d, generator=g) * torch.exp(2 * torch.randn(B, H, N, 1, generator=g))
    return x.to(torch.bfloat16)


def _empty(blocks, page, H, d, e4m3):
    kind = torch.uint8 if e4m3 else torch.bfloat16
    pages = [torch.full((blocks, page, H, d), 7, dtype=kind, device="cuda") for _ in range(2)]
    ds = [torch.full((blocks, H, page), -3.0, device="cuda") if e4m3 else None for _ in range(2)]
    return pages, ds


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,H,N,d,page", [(1, 1, 1, 128, 64), (3, 2, 37, 64, 16), (2, 8, 100, 80, 48),
                                          (2, 3, 65, 256, 1), (1, 4, 31, 16, 7), (5, 1, 64, 208, 128)])
def test_write_bit_for_bit(B, H, N, d, page, e4m3):
    k, v = _rows(B, H, N, d), _rows(B, H, N, d, seed=1)
    k[0, 0, 0] = 0                                      # an all-zero row
    blocks = -(-B * N // page) + 2
    slots = torch.randperm(blocks * page, generator=torch.Generator().manual_seed(3))[:B * N].reshape(B, N)
    if N > 2:
        slots[0, 1] = -1                                # padding
    (kp, vp), (kd, vd) = _empty(blocks, page, H, d, e4m3)
    want = [x.cpu().clone() for x in (kp, vp)]
    want_d = [None if x is None else x.cpu().clone() for x in (kd, vd)]
    # token-major values: strides other than the keys'
    ea.attn_cache_write(k.cuda(), v.transpose(1, 2).contiguous().cuda().transpose(1, 2), kp, vp,
                        slots.cuda(), kd, vd)
    live = slots.reshape(-1) >= 0
    at = slots.reshape(-1)[live]
    for x, pages, ds in zip((k, v), want, want_d):
        rows = x.transpose(1, 2).reshape(-1, H, d)[live]
        if e4m3:
            rows, scale = quantize(rows)
            ds[at // page, :, at % page] = scale
        pages.view(-1, H, d)[at] = rows
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    for got, ref in zip((kp, vp), want):                # rows no slot names stay as they were
        assert torch.equal(got.cpu().view(torch.uint8), ref.view(torch.uint8))
    if e4m3:
        for got, ref in zip((kd, vd), want_d):
            assert torch.equal(got.cpu(), ref)


def test_write_error_against_the_values():
    """|code * descale - x| <= half a step (2^-4 |x|, or 2^-10 descale below
    the normal codes) and the fp32 roundings of 448 / a, the product and the descale."""
    k = _rows(2, 4, 333, 128)
    (kp, vp), (kd, vd) = _empty(11, 64, 4, 128, True)
    slots = torch.arange(666).reshape(2, 333).cuda()
    ea.attn_cache_write(k.cuda(), k.cuda(), kp, vp, slots, kd, vd)
    x = k.transpose(1, 2).reshape(666, 4, 128).double()
    scale = kd.cpu().transpose(1, 2).reshape(-1, 4)[:666].double()[..., None]
    val = kp.cpu().view(torch.float8_e4m3fn).double().reshape(-1, 4, 128)[:666] * scale
    assert ((val - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * scale) + 2.0 ** -21 * x.abs()).all()


def test_write_special_values():
    """Tiny, huge, infinite and NaN rows; each stays in its own row."""
    d = 64
    x = torch.zeros(1, 1, 7, d, dtype=torch.bfloat16)
    x[0, 0, 0] = 1e-38                                  # below the smallest scale's maximum
    x[0, 0, 1, 3] = 1e-40                               # subnormal
    x[0, 0, 2] = 3e38
    x[0, 0, 3, :] = 1.0
    x[0, 0, 3, 5] = float("nan")
    x[0, 0, 4, :] = 1.0
    x[0, 0, 4, 6] = float("inf")
    x[0, 0, 5, :] = float("nan")
    x[0, 0, 6, :] = torch.linspace(-3, 3, d).to(torch.bfloat16)
    (kp, vp), (kd, vd) = _empty(1, 16, 1, d, True)
    ea.attn_cache_write(x.cuda(), x.cuda(), kp, vp, torch.arange(7).cuda().reshape(1, 7), kd, vd)
    codes, scale = quantize(x[0, 0])
    got = kp[0, :7, 0].cpu()
    f8 = got.view(torch.float8_e4m3fn).float()
    assert torch.equal(kd[0, 0, :7].cpu(), scale)
    for r in (0, 1, 2, 6):
        assert torch.equal(got[r], codes[r]) and torch.isfinite(scale[r])
    assert torch.isnan(f8[3, 5]) and torch.equal(f8[3, :5], torch.full((5,), 448.0))
    assert torch.isnan(f8[4] * kd[0, 0, 4].cpu()).all()
    assert torch.isnan(f8[5]).all() and kd[0, 0, 5] == 1


def test_write_bad_slots_are_skipped_and_reported():
    x = _rows(1, 2, 5, 32).cuda()
    (kp, vp), _ = _empty(2, 16, 2, 32, False)
    before = kp.clone()
    assert ea.attn_last_device_error() == 0
    ea.attn_cache_write(x, x, kp, vp, torch.tensor([[32, -2, 2 ** 40, 5, -1]]).cuda())
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    before[0, 5] = x[0, :, 3]
    assert torch.equal(kp, before) and torch.equal(vp[0, 5], x[0, :, 3])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths,H,d,page", [
    ([1], 1, 128, 64), ([0, 5, 0, 17, 64], 2, 80, 16), ([100, 1, 999], 4, 128, 48), ([33], 3, 256, 5)])
def test_read(lengths, H, d, page, e4m3, out):
    c = Cache(lengths, H, d, page, e4m3, seed=7, outliers=True)
    (kp, vp, table, _), (kd, vd) = c.on("cuda")
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32) + 2       # rows before and behind stay
    total = int(cu[-1]) + 3
    ko = torch.full((total, H, d), 9.0, dtype=out, device="cuda")
    vo = ko.clone()
    ea.attn_cache_read(kp, vp, table, cu.cuda(), ko, vo, kd, vd)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    for which, got in (("k", ko.cpu()), ("v", vo.cpu())):
        assert (got[:2] == 9).all() and (got[int(cu[-1]):] == 9).all()
        for b, n in enumerate(lengths):
            ref = c.values(which, b)
            diff = (got[int(cu[b]):int(cu[b + 1])].double() - ref).abs()
            assert (diff <= (HALF[out] + 2.0 ** -24) * 1.01 * ref.abs()).all()


def test_read_bad_offsets_and_pages():
    c = Cache([64, 64], 1, 32, 32, seed=1)
    (kp, vp, table, _), _ = c.on("cuda")
    k, v = torch.full((140, 1, 32), 9.0, device="cuda"), torch.full((140, 1, 32), 9.0, device="cuda")
    # the first sequence is longer than its table; the second is fine
    ea.attn_cache_read(kp, vp, table, torch.tensor([0, 70, 134], dtype=torch.int32).cuda(), k, v)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == ea.ATTN_ERR_INVALID_ARG
    assert (k[:70] == 9).all() and (k[134:] == 9).all()
    assert torch.equal(k[70:134].cpu().double(), c.values("k", 1))
    for cu in ([-3, 61, 125], [0, 64, 200], [0, 64, 30]):
        k.fill_(9.0)
        ea.attn_cache_read(kp, vp, table, torch.tensor(cu, dtype=torch.int32).cuda(), k, v)
        torch.cuda.synchronize()
        ea.attn_last_device_error()
        if cu[0] == 0:
            assert torch.equal(k[:30].cpu().double(), c.values("k", 0)[:30])
    table[1, 0] = -1                                       # an entry that names no page
    k.fill_(9.0)
    ea.attn_cache_read(kp, vp, table, torch.tensor([0, 64, 128], dtype=torch.int32).cuda(), k, v)
    torch.cuda.synchronize()
    assert ea.attn_last_device_error() == 0
    assert (k[64:96] == 0).all() and torch.equal(k[96:128].cpu().double(), c.values("k", 1)[32:])


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_past_32_bits(e4m3):
    """Pages past 2^32 elements of the cache: write there, read back."""
    H, d, page = 8, 128, 64
    blocks = 2 ** 32 // (H * d * page) + 3
    kind = torch.uint8 if e4m3 else torch.bfloat16
    kp = torch.empty(blocks, page, H, d, dtype=kind, device="cuda")
    ds = torch.empty(blocks, H, page, device="cuda") if e4m3 else None
    x = _rows(1, H, 70, d).cuda()
    first = (blocks - 2) * page
    ea.attn_cache_write(x, x, kp, kp, (first + torch.arange(70)).reshape(1, 70).cuda(), ds, ds)
    table = torch.tensor([[blocks - 2, blocks - 1]], dtype=torch.int32).cuda()
    k, _ = ea.cache_read(kp, kp, table, torch.tensor([0, 70], dtype=torch.int32).cuda(), 70, ds, ds)
    rows = x[0].transpose(0, 1).cpu()
    if e4m3:
        codes, scale = quantize(rows)
        rows = (codes.view(torch.float8_e4m3fn).float() * scale[..., None]).to(torch.bfloat16)
    assert torch.equal(k.cpu(), rows)
