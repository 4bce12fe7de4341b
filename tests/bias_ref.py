"""Plain 64-bit forms of attention with a relative position bias, its gradients,
and the paged cache's tables, with the error bounds their tests share (CPU, torch
double precision)."""
import math

import torch

U16, U32 = 2.0 ** -8, 2.0 ** -24     # half a step of bf16 and of fp32, relative


def bucket(r, n, D):
    """Bucket of a distance r >= 0 back among n of a direction, in whole numbers."""
    e = n // 2
    if r < e:
        return r
    s, k = n - e, 0
    while k + 1 < s and r ** s * e ** (k + 1) >= D ** (k + 1) * e ** s:
        k += 1
    return e + k


def bias64(table, buckets, first, n, m):
    """[H, n, m]: the bias of query i and key j; what is below -1e6 is -inf."""
    r = torch.arange(m) - (torch.arange(n)[:, None] + m - n)
    b = buckets.cpu().long()[(r - first).clamp(0, len(buckets) - 1)]
    t = table.cpu().double()
    t = torch.where(t < -1e6, torch.full_like(t, -math.inf), t)
    return t.t()[:, b], b


class Problem:
    """One dense problem: q [Hq, n, d], k, v [Hkv, m, d] (any float type)."""

    def __init__(self, q, k, v, table, buckets, first, causal=False, scale=None):
        self.d = q.shape[-1]
        self.scale = self.d ** -0.5 if scale is None else scale
        G = q.shape[0] // k.shape[0]
        self.G = G
        self.q, self.k, self.v = q.double(), k.double().repeat_interleave(G, 0), v.double().repeat_interleave(G, 0)
        n, m = q.shape[1], k.shape[1]
        self.n, self.m = n, m
        bias, self.buckets = bias64(table, buckets, first, n, m)
        x = self.q @ self.k.transpose(1, 2) * self.scale + bias
        if causal:
            x = x.masked_fill(torch.ones(n, m, dtype=torch.bool).triu(m - n + 1), -math.inf)
        self.x = x
        top = x.amax(-1, keepdim=True)
        empty = top == -math.inf
        p = torch.exp(x - torch.where(empty, torch.zeros_like(top), top))
        total = p.sum(-1, keepdim=True)
        self.p = p / total.masked_fill(empty, 1.0)
        self.lse = torch.where(empty, top, torch.log(total) + top).squeeze(-1)
        self.o = self.p @ self.v
        # a score's error in fp32: d products summed, the scale, the bias added, and
        # the exponent's own roundings at the size of the row's scores
        live = torch.where(x == -math.inf, torch.zeros_like(x), x)
        dot = (self.q.abs() @ self.k.abs().transpose(1, 2)).amax(-1) * self.scale
        self.dx = U32 * (self.d * dot + 8 * live.abs().amax(-1) + 8)

    def check_forward(self, o, lse):
        """P is rounded to bf16 (half a step each), the normaliser by at most as
        much, and a weight is off by the score's error; O's own rounding comes on
        top.  LSE: the scores' error, and N / 4 + 64 additions of fp32."""
        rounding = U16 * self.o.abs() if o.dtype == torch.bfloat16 else 0.0
        bound = (2 * U16 + 4 * self.dx)[..., None] * (self.p @ self.v.abs()) + rounding + 1e-30
        err = (o.cpu().double() - self.o).abs()
        assert (err <= bound).all(), float((err / bound).max())
        lse = lse.cpu().double()
        assert torch.equal(lse == -math.inf, self.lse == -math.inf)
        err = torch.where(lse == -math.inf, 0.0, lse - self.lse).abs()
        bound = 2 * self.dx + U32 * (self.m / 4 + 64 + 4 * torch.nan_to_num(self.lse, neginf=0.0).abs())
        assert (err <= bound).all(), float((err / bound).max())

    def gradients(self, o, dout, lse, num_buckets):
        """(dq, dk, dv, dtable) of these o and lse, and a bound for each: P and dS
        are rounded to bf16 for the products (not for the table), P is off by the
        score's error, dP - D by d fp32 additions of products the size of |dO| |V|
        (and |dO| |O|); sums over diagonals in fp32, at most 2^10 deep."""
        o, dout, lse = o.cpu().double(), dout.cpu().double(), lse.cpu().double()
        p = torch.exp(self.x - torch.where(lse == -math.inf, math.inf, lse)[..., None])
        dp = dout @ self.v.transpose(1, 2)
        D = (dout * o).sum(-1, keepdim=True)
        ds = p * (dp - D)
        size = dout.abs() @ self.v.abs().transpose(1, 2) + (dout.abs() * o.abs()).sum(-1, keepdim=True)
        e = (4 * self.dx)[..., None] * ds.abs() + U32 * self.d * p * size   # of an unrounded dS
        e16 = e + U16 * ds.abs() * (1 + U16)

        def group(t):
            return t.view(-1, self.G, *t.shape[1:]).sum(1)
        s = self.scale
        grads = [ds @ self.k * s, group(ds.transpose(1, 2) @ self.q) * s, group(p.transpose(1, 2) @ dout)]
        bounds = [e16 @ self.k.abs() * s, group(e16.transpose(1, 2) @ self.q.abs()) * s,
                  group((p * (U16 + 4 * self.dx[..., None])).transpose(1, 2) @ dout.abs())]
        H = p.shape[0]
        at = self.buckets.reshape(-1)

        def per_bucket(t):
            return torch.zeros(num_buckets, H, dtype=torch.float64).index_add_(0, at, t.reshape(H, -1).t())
        grads.append(per_bucket(ds))
        bounds.append(per_bucket(e + 1024 * U32 * ds.abs()))
        return grads, bounds


def check_gradients(got, grads, bounds):
    for name, g, want, bound in zip(("dq", "dk", "dv", "dtable"), got, grads, bounds):
        rounding = (U16 if g.dtype == torch.bfloat16 else 2 * U32) * want.abs()
        err = (g.cpu().double() - want).abs()
        ok = err <= bound * 1.01 + rounding + 1e-30
        assert ok.all(), (name, float((err / (bound + rounding + 1e-30)).max()))


class Pages:
    """The pool and the tables in plain Python: extend and trim as specified."""

    def __init__(self, num_blocks, B, max_blocks, page):
        self.free = list(range(num_blocks - 1, -1, -1))
        self.num_blocks, self.page, self.max_blocks = num_blocks, page, max_blocks
        self.table = [[-1] * max_blocks for _ in range(B)]
        self.len = [0] * B

    def _pages(self, n):
        return -(-n // self.page)

    def extend(self, new, width=None):
        """(slots, positions, granted) as lists of rows, one list a request."""
        out, ran_out, upto, count = [], False, 0, len(self.free)
        for b, add in enumerate(new):
            n = self.len[b]
            if add < 0 or n + add > self.max_blocks * self.page or (width and add > width):
                add = 0
            need = self._pages(n + add) - self._pages(n)
            upto += need
            ran_out = need > 0 and (ran_out or upto > count)
            ok = need == 0 or upto <= count
            if ok:
                for i in range(need):
                    self.table[b][self._pages(n) + i] = self.free.pop()
                self.len[b] = n + add
            row = [self.table[b][p // self.page] * self.page + p % self.page if ok else -1
                   for p in range(n, n + add)]
            out.append((row, list(range(n, n + add)), add if ok else 0))
        return out

    def trim(self, keep):
        back = []
        for b, k in enumerate(keep):
            k = max(0, min(k, self.len[b]))
            back += self.table[b][self._pages(k):self._pages(self.len[b])]
            self.len[b] = k
        self.free += back[::-1]
