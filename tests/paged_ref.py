"""Plain 64-bit forms of the position, cache and tree-attention operators, and
the inputs their tests share (CPU tensors, torch double precision)."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
        torch.float8_e4m3fn: 2.0 ** -4}


def rope64(x, positions, inv_freq, interleaved=False, inverse=False, magnitude=1.0):
    """x [B,H,N,d] -> (fp64 result, |a| + |b| of every element's pair)."""
    x = x.double()
    r = 2 * inv_freq.numel()
    if positions.ndim == 1:
        positions = positions[None].expand(x.shape[0], -1)
    th = positions.double()[:, None, :, None] * inv_freq
    c, s = torch.cos(th), torch.sin(th) * (-1 if inverse else 1)
    y, size = x.clone(), torch.zeros_like(x)
    ia = torch.arange(0, r, 2) if interleaved else torch.arange(r // 2)
    ib = ia + 1 if interleaved else ia + r // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = magnitude * (a * c - b * s)
    y[..., ib] = magnitude * (a * s + b * c)
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size * abs(magnitude)


def quantize(x):
    """bf16 rows [..., d] -> (uint8 E4M3 codes, fp32 descale [...]), in fp32."""
    x = x.float()
    amax = torch.where(x.isnan(), torch.zeros_like(x), x.abs()).amax(-1)
    a = amax.clamp(min=2.0 ** -100)
    # (448.0 / a would be a.reciprocal() * 448: 448 / 5.75 is 0x1.37a6f4p+6, that gives 0x1.37a6f6p+6)
    scale = torch.where(amax > 0, torch.full_like(a, 448.0) / a, torch.ones_like(a))
    codes = (x * scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, torch.where(amax > 0, a / 448.0, torch.ones_like(a))


class Cache:
    """A paged cache with sequences of the given lengths on scattered pages.
    Everything outside the sequences is NaN.  k, v: [B][len, Hkv, d] bf16."""

    def __init__(self, lengths, Hkv, d, page, e4m3=False, seed=0, max_blocks=None, k=None, v=None,
                 outliers=False):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.page, self.e4m3 = list(lengths), page, e4m3
        B = len(lengths)
        need = [-(-n // page) for n in lengths]
        width = max_blocks or max(max(need), 1)
        total = sum(need) + 2
        perm = torch.randperm(total, generator=g)
        size = torch.exp(torch.randn(max(sum(lengths), 1), 1, 1, generator=g)) if outliers else 1.0

        def rows():
            x = torch.randn(max(sum(lengths), 1), Hkv, d, generator=g) * size
            return list(x.to(torch.bfloat16)[:sum(lengths)].split(list(lengths)))
        self.k, self.v = k or rows(), v or rows()
        self.table = torch.full((B, width), 2 ** 30, dtype=torch.int32)   # names no page
        kind = torch.uint8 if e4m3 else torch.bfloat16
        fill = 0x7F if e4m3 else float("nan")
        self.k_pages = torch.full((total, page, Hkv, d), fill, dtype=kind)
        self.v_pages = self.k_pages.clone()
        self.k_descale = self.v_descale = None
        if e4m3:
            self.k_descale = torch.full((total, Hkv, page), float("nan"))
            self.v_descale = self.k_descale.clone()
        at = 0
        self.slots = []
        for b, n in enumerate(lengths):
            ids = perm[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = ids.to(torch.int32)
            pos = torch.arange(n)
            slot = ids[pos // page] * page + pos % page if n else pos
            self.slots.append(slot)
            for x, pages, descale in ((self.k[b], self.k_pages, self.k_descale),
                                      (self.v[b], self.v_pages, self.v_descale)):
                if e4m3:
                    x, ds = quantize(x)
                    descale[slot // page, :, slot % page] = ds
                pages.view(-1, Hkv, d)[slot] = x
        self.seqlens = torch.tensor(list(lengths), dtype=torch.int32)

    def values(self, which, b):
        """The fp64 values [len, Hkv, d] of sequence b's cached rows."""
        pages, descale = (self.k_pages, self.k_descale) if which == "k" else (self.v_pages, self.v_descale)
        slot = self.slots[b]
        x = pages.reshape(-1, *pages.shape[2:])[slot]
        if not self.e4m3:
            return x.double()
        return x.view(torch.float8_e4m3fn).double() * descale[slot // self.page, :, slot % self.page].double()[..., None]

    def on(self, dev):
        """k_pages, v_pages, block_table, seqlens, and the descales, on a device."""
        d = [None if x is None else x.to(dev) for x in (self.k_descale, self.v_descale)]
        return [x.to(dev) for x in (self.k_pages, self.v_pages, self.table, self.seqlens)], d


def random_trees(B, T, seed):
    """bool [B,T,T]: each token sees itself and its ancestors."""
    g = torch.Generator().manual_seed(seed)
    m = torch.zeros(B, T, T, dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            parent = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            if parent >= 0:
                m[b, t] = m[b, parent]
            m[b, t, t] = True
    return m


def tree64(q, cache, mask=None, q_lens=None, scale=None):
    """(O, LSE, bound): fp64 tree attention, and for each O element sum_j p_j |v_j|,
    for each row the size of the rounding of its scores (see score_eps)."""
    B, Hq, T, d = q.shape
    o = torch.zeros(B, Hq, T, d, dtype=torch.float64)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64)
    size = torch.zeros_like(o)
    eps = torch.zeros(B, Hq, T, dtype=torch.float64)
    scale = d ** -0.5 if scale is None else scale
    for b in range(B):
        n = T if q_lens is None else int(q_lens[b])
        k, v = cache.values("k", b), cache.values("v", b)
        L, Hkv = k.shape[0], k.shape[1]
        if n == 0:
            continue
        see = torch.ones(n, L, dtype=torch.bool)
        see[:, L - n:] = torch.tril(torch.ones(n, n, dtype=torch.bool)) if mask is None else mask[b, :n, :n]
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            qd = q[b, h, :n].double()
            for t in range(n):
                js = see[t].nonzero().squeeze(1)     # (unseen keys take no part, NaN or not)
                if js.numel() == 0:
                    continue
                s = scale * (k[js, kv] @ qd[t])
                z = torch.logsumexp(s, 0)
                p = torch.exp(s - z)
                o[b, h, t] = p @ v[js, kv]
                size[b, h, t] = p @ v[js, kv].abs()
                lse[b, h, t] = z
                # fp32 accumulation of d products (any order): d * 2^-23 of the sum of |q||k|
                eps[b, h, t] = d * 2.0 ** -23 * scale * (k[js, kv].abs() @ qd[t].abs()).max()
                if cache.e4m3:
                    # with many rows Q is the sum of two E4M3 terms, its row scaled to a largest
                    # value in [2^7, 2^8): 8 bits from 2^-2 up are exact (the residual of 4 of them
                    # has 4, none below 2^-9), below that off by at most 2^-10, 2^-17 of the largest
                    a = qd[t].abs()
                    small = 2.0 ** -17 * a.max() * (a < 2.0 ** -9 * a.max())
                    eps[b, h, t] += scale * (k[js, kv].abs() @ small).max()
    return o, lse, size, eps


def check_tree(o, lse, ref, e4m3, o_dtype):
    """O and LSE of the kernel against tree64's result.

    With weights off by a factor 1 + delta_j, |delta_j| <= u (P's rounding to
    bf16 2^-8, or for E4M3 to fp16 2^-11) + e (scores: eps; 2^x: 2^-21), the
    quotient sum w v / sum w is off by at most 2 (u + e) sum p |v|, the sums
    and merges by a few 2^-23 of it, and the output's rounding adds 2^-8 |O| (bf16) or 2^-24."""
    ro, rl, size, eps = ref
    # E4M3 with many rows: V enters as fp16(code * fp16(vd / F)) and P as fp16, each
    # rounding 2^-11, while the sum that divides is of unrounded P: 3 * 2^-11 of
    # sum p |v|, where 2 u is used below
    u = 1.5 * 2.0 ** -11 if e4m3 else 2.0 ** -8
    o, lse = o.double().cpu(), lse.double().cpu()
    tol = (2 * (u + eps[..., None] + 2.0 ** -21) + 2.0 ** -19) * size * 1.02 + HALF[o_dtype] * ro.abs() + 1e-30
    assert ((o - ro).abs() <= tol).all(), ((o - ro).abs() - tol).max()
    dead = rl == -math.inf
    assert torch.equal(lse == -math.inf, dead)
    assert (o[dead] == 0).all()
    live = ~dead
    ltol = eps + 2.0 ** -19 * (1 + rl.abs())
    assert ((lse - rl).abs()[live] <= ltol[live]).all(), ((lse - rl).abs()[live] - ltol[live]).max()
