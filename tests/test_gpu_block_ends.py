"""Packed arrays that end where a 2 MB block of memory does: their tensor maps begin
lower (encode_tmap_ragged), and the results are those of the same arrays elsewhere."""
import pytest
import torch

import exact_attention_14_gb300 as ea

pytestmark = pytest.mark.gpu

BLOCK = 2 << 20
LENS = ([5, 1, 1, 0, 130], [7, 64, 148, 64, 131])


def _at_end(t, back=0):
    """A copy of t whose last byte is `back` bytes before the end of a block."""
    n = t.numel() * t.element_size()
    buf = torch.zeros(3 * BLOCK, dtype=torch.uint8, device="cuda")
    end = (-buf.data_ptr()) % BLOCK + BLOCK - back
    x = buf[end - n:end].view(t.dtype).view(t.shape)
    x.copy_(t)
    assert (x.data_ptr() + n + back) % BLOCK == 0 and x.is_contiguous()
    return x


def _inputs(Hq, Hkv, d):
    g = torch.Generator().manual_seed(d)
    cu = [torch.tensor([0] + n).cumsum(0).to(torch.int32).cuda() for n in LENS]
    tq, tk = sum(LENS[0]), sum(LENS[1])
    q, dout = (torch.randn(tq, Hq, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    k, v = (torch.randn(tk, Hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    return q, k, v, dout, cu


@pytest.mark.parametrize("back", [0, 16, 4096 + 16, 200000 // 16 * 16])
@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 16), (2, 1, 80), (1, 1, 64), (2, 2, 128), (1, 1, 136), (1, 1, 256)])
def test_same_bits_at_the_end_of_a_block(Hq, Hkv, d, back):
    q, k, v, dout, (cq, ck) = _inputs(Hq, Hkv, d)
    mq, mk = max(LENS[0]), max(LENS[1])
    qe, ke, ve, de = (_at_end(t, back) for t in (q, k, v, dout))
    for causal in (False, True):
        o, lse = ea.forward_varlen(q, k, v, cq, ck, mq, mk, causal=causal)
        oe, lse_e = _at_end(torch.zeros_like(o), back), torch.empty_like(lse)
        ea.attn_fwd_varlen(qe, ke, ve, oe, cq, ck, mq, mk, lse_e, causal=causal)
        assert torch.equal(o, oe) and torch.equal(lse, lse_e)
        for kind in (torch.bfloat16, torch.float32):
            want = ea.backward_varlen(q, k, v, o, dout, lse, cq, ck, mq, mk, causal=causal, grad_dtype=kind)
            got = [_at_end(torch.zeros_like(t), back) for t in want]
            ea.attn_bwd_varlen(qe, ke, ve, oe, de, lse, *got, cq, ck, mq, mk, causal=causal)
            assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert ea.attn_last_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 80), (1, 1, 64), (2, 2, 128)])
def test_the_same_with_a_bias(Hq, Hkv, d):
    q, k, v, dout, (cq, ck) = _inputs(Hq, Hkv, d)
    ids, first = ea.bias_buckets(32, 128)
    table = torch.randn(32, Hq, generator=torch.Generator().manual_seed(1)).cuda()
    mq, mk = max(LENS[0]), max(LENS[1])
    qe, ke, ve, de = (_at_end(t) for t in (q, k, v, dout))
    o, lse = ea.forward_varlen_bias(q, k, v, cq, ck, mq, mk, table, ids, first, causal=True)
    oe, lse_e = ea.forward_varlen_bias(qe, ke, ve, cq, ck, mq, mk, table, ids, first, causal=True)
    assert torch.equal(o, oe) and torch.equal(lse, lse_e)
    want = ea.backward_varlen_bias(q, k, v, o, dout, lse, cq, ck, mq, mk, table, ids, first, causal=True)
    got = [_at_end(torch.zeros_like(t)) for t in want]
    ea.attn_bwd_varlen_bias(qe, ke, ve, oe, de, lse, table, ids, first, *got, cq, ck, mq, mk, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert ea.attn_last_device_error() == 0
