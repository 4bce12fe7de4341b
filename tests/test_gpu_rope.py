"""attn_rope on the GPU against the 64-bit rotation."""
import pytest
import torch

import exact_attention_14_gb300 as ea
from paged_ref import HALF, rope64

pytestmark = pytest.mark.gpu


def _x(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _close(got, x, positions, f, dtype, **kw):
    """cos / sin are within 6.6 * 2^-24 of the exact ones (argument 1.6, sincospi
    2, magnitude 1, product and sum 1 each): 2^-21 of |a| + |b|, then the output's rounding."""
    ref, size = rope64(x, positions, f, **kw)
    tol = HALF[dtype] * 1.01 * ref.abs() + 2.0 ** -21 * size
    assert ((got.double().cpu() - ref).abs() <= tol).all()


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,inter", [
    (2, 37, 4, 2, 128, 128, False), (1, 1, 32, 8, 128, 128, False), (3, 5, 3, 3, 64, 64, True),
    (2, 65, 8, 1, 96, 40, True), (2, 65, 8, 1, 96, 40, False), (1, 300, 2, 2, 80, 20, False),
    (1, 33, 2, 1, 256, 256, False), (1, 33, 2, 1, 256, 250, True), (2, 9, 2, 1, 8, 2, False),
    (2, 9, 2, 1, 8, 6, True), (1, 7, 5, 5, 200, 48, False), (1, 1000, 40, 8, 128, 64, False),
])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("dt,odt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                    (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_matches_the_rotation(B, N, Hq, Hkv, d, rot, inter, inverse, dt, odt):
    q, k = _x(B, Hq, N, d, dtype=dt), _x(B, Hkv, N, d, seed=1, dtype=dt)
    pos = torch.randint(0, 1 << 20, (B, N), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    f, mag = ea.rope_frequencies(rot, 10000.0, scaling="by_parts", factor=4.0, original_len=4096,
                                 device="cpu")
    qo, ko = ea.rope(q.cuda(), k.cuda(), pos.cuda(), f.cuda(), interleaved=inter, magnitude=mag,
                     out_dtype=odt, inverse=inverse)
    assert qo.dtype == odt and qo.shape == q.shape and ko.shape == k.shape
    _close(qo, q, pos, f, odt, interleaved=inter, inverse=inverse, magnitude=mag)
    _close(ko, k, pos, f, odt, interleaved=inter, inverse=inverse, magnitude=mag)


@pytest.mark.parametrize("positions", [
    [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 999999937, -123456789]])
def test_any_32_bit_position_and_large_frequencies(positions):
    """The phase is exact: no loss at the far end, nor for frequencies of several turns."""
    pos = torch.tensor(positions, dtype=torch.int32)
    f = torch.tensor([1.0, 3.0, 0.5, 1e-9, 7.0, -2.25, 100.0, 0.0], dtype=torch.float64)
    x = _x(1, 2, len(positions), 16, dtype=torch.float32)
    got, _ = ea.rope(x.cuda(), None, pos.cuda(), f.cuda())
    # (pos * f in fp64 is exact for these f but 1e-9, whose angle is small)
    _close(got, x, pos, f, torch.float32)


@pytest.mark.parametrize("inter,rot", [(False, 128), (False, 36), (True, 128), (True, 36)])
def test_layouts_in_place_and_strided(inter, rot):
    """Token-major projections, packed rows, shared positions, in place."""
    B, N, Hq, Hkv, d = 2, 19, 6, 2, 128
    both = _x(B, N, Hq + Hkv, d).cuda()
    pos = torch.arange(100, 100 + N, dtype=torch.int32, device="cuda")
    f, _ = ea.rope_frequencies(rot)
    q, k = both[:, :, :Hq].transpose(1, 2), both[:, :, Hq:].transpose(1, 2)
    want_q, want_k = ea.rope(q.contiguous(), k.contiguous(), pos[None].expand(B, N), f, interleaved=inter)
    got_q, got_k = ea.rope(q, k, pos, f, interleaved=inter)
    assert torch.equal(got_q, want_q) and torch.equal(got_k, want_k)
    # packed [total, H, d]
    pq, pk = ea.rope(both[0, :, :Hq], both[0, :, Hq:], pos, f, interleaved=inter)
    assert torch.equal(pq, want_q[0].transpose(0, 1)) and torch.equal(pk, want_k[0].transpose(0, 1))
    # in place, in the projection's rows; the columns past rotary_dim stay
    ea.attn_rope(q, k, q, k, pos, f, interleaved=inter)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)


def test_inverse_is_the_transpose():
    """<R x, y> = <x, R^T y>, and R^T R = magnitude^2: the gradient against the formula."""
    B, H, N, d = 1, 2, 50, 96
    x, y = _x(B, H, N, d, dtype=torch.float32).cuda(), _x(B, H, N, d, seed=4, dtype=torch.float32).cuda()
    pos = torch.arange(N, dtype=torch.int32, device="cuda") * 1000
    f, _ = ea.rope_frequencies(64)
    rx, _ = ea.rope(x, None, pos, f, magnitude=1.5)
    ry, none = ea.rope_backward(y, None, pos, f, magnitude=1.5)
    assert none is None
    a, b = (rx.double() * y.double()).sum(-1), (x.double() * ry.double()).sum(-1)
    # d products, each factor within 2^-21 (|a| + |b|) * 1.5
    tol = 2 * 1.5 * 2.0 ** -21 * 2 * x.double().norm(dim=-1) * y.double().norm(dim=-1) * d ** 0.5
    assert ((a - b).abs() <= tol).all()
    # differences: f(x) = <R x, y> is linear, so its slope is R^T y itself
    h = 2.0 ** -3
    for col in (0, 31, 40, 63, 64, 95):
        x2 = x.clone()
        x2[..., col] += h
        r2, _ = ea.rope(x2, None, pos, f, magnitude=1.5)
        slope = ((r2.double() - rx.double()) * y.double()).sum(-1) / (x2[..., col].double() - x[..., col].double())
        tol = 4 * 2.0 ** -21 * 1.5 * (x.double().abs().amax(-1) + h) * y.double().abs().sum(-1) / h
        assert ((slope - ry[..., col].double()).abs() <= tol).all()


def test_stream_graph_and_far_rows():
    d, N = 128, 64
    x = _x(1, 4, N, d).cuda()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    f, _ = ea.rope_frequencies(d)
    want, _ = ea.rope(x, None, pos, f)
    out = torch.zeros_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ea.attn_rope(x, None, out, None, pos, f)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    x.neg_()
    pos += 5
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ea.rope(x, None, pos, f)[0])
    # rows past 2^31 elements from the base
    big = torch.empty(2 ** 31 // (4 * d) + 70, 4, d, dtype=torch.bfloat16, device="cuda")
    tail = big[-64:]
    tail.copy_(x[0].transpose(0, 1))
    view = big.as_strided((2, 64, 4, d), ((big.shape[0] - 64) * 4 * d, 4 * d, d, 1)).transpose(1, 2)
    view[0].copy_(x[0])
    got, _ = ea.rope(view, None, pos, f)
    assert torch.equal(got[1], got[0])
