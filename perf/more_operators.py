"""Attention with a learned relative position bias, and the paged cache's tables, as they are measured.

Four kinds of case, told apart by ``op``:

  forward   softmax(scale Q K^T + bias) V and its logsumexp, dense or packed
  backward  the gradients of Q, K, V and of the bias table, dense or packed
  decode    one new token a sequence over a paged cache, with the bias
  pages     block tables and cache slots of a step's new tokens built from the
            requests' lengths (and the pages taken back again)

The bias of query head h at relative distance r = key position - query position
(the last query stands at the last key) is table[buckets[clamp(r - first)], h].

With ``own`` false, ``run`` computes an operator with elementary torch
operations in 32 bits (sums over whole diagonals in 64); with ``own`` true it
calls the library.  ``exact`` computes the same in 64 bits.
"""
import math

import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest call: one head, 256 positions, a small model's head width
        dict(name="forward_tiny", op="forward", B=1, Hq=1, Hkv=1, Nq=256, Nk=256, d=64, causal=False,
             buckets=32, distance=128, bf16=False),
        # an encoder layer's forward: 4 x 2048 positions, both directions
        dict(name="forward_encoder", op="forward", B=4, Hq=16, Hkv=16, Nq=2048, Nk=2048, d=128,
             causal=False, buckets=32, distance=128, bf16=False),
        # a decoder's prefill with grouped heads and a bf16 table: the largest forward
        dict(name="forward_grouped", op="forward", B=8, Hq=32, Hkv=8, Nq=4096, Nk=4096, d=128,
             causal=True, buckets=32, distance=128, bf16=True),
        # packed prompts of odd lengths, each after a cached prefix, buckets over 1024 positions
        dict(name="forward_packed_odd", op="forward", B=13, Hq=12, Hkv=4, lo=1, hi=2501, prefix=131,
             d=80, causal=True, buckets=64, distance=1024, bf16=False),
        # gradients at odd sizes, more keys than queries, grouped heads
        dict(name="backward_odd", op="backward", B=3, Hq=6, Hkv=2, Nq=333, Nk=517, d=96, causal=True,
             buckets=32, distance=128, bf16=False),
        # an encoder layer's backward
        dict(name="backward_encoder", op="backward", B=4, Hq=16, Hkv=16, Nq=2048, Nk=2048, d=128,
             causal=False, buckets=32, distance=128, bf16=False),
        # the packed prefill workload's backward, buckets over 2048 positions: the largest
        dict(name="backward_packed", op="backward", B=16, Hq=16, Hkv=16, lo=256, hi=4096, prefix=0,
             d=128, causal=True, buckets=128, distance=2048, bf16=True),
        # a few short, odd contexts: latency
        dict(name="decode_small", op="decode", B=3, Hq=8, Hkv=2, d=96, page=64, lo=40, hi=777,
             buckets=32, distance=128, bf16=False),
        # the decode workload
        dict(name="decode_long", op="decode", B=16, Hq=32, Hkv=8, d=128, page=64, lo=1024, hi=32768,
             buckets=32, distance=128, bf16=True),
        # one decode step's new tokens of 16 requests
        dict(name="pages_step", op="pages", B=16, page=64, lo=1024, hi=32767, new_lo=1, new_hi=1, T=1,
             short=0.0),
        # a few drafted tokens a request, padded rows, a pool that runs out on the way
        dict(name="pages_drafts_short", op="pages", B=61, page=16, lo=0, hi=5003, new_lo=0, new_hi=7,
             T=7, short=0.4),
        # 512 prompts admitted at once: a million tokens in 16-token pages
        dict(name="pages_prompts", op="pages", B=512, page=16, lo=0, hi=0, new_lo=17, new_hi=4096, T=0,
             short=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "decode", "pages"])
    if op == "pages":
        page = rng.choice([1, 16, 48, 64, 128, 256])
        B = _log_int(rng, 1, 1024)
        T = rng.choice([0, 0, 1, _log_int(rng, 1, 64)])
        new_hi = T if T else max(1, min(_log_int(rng, 1, 8192), (1 << 20) // B))
        hi = _log_int(rng, 1, 32768 if page > 1 else 2048)
        return dict(op="pages", B=B, page=page, lo=rng.randint(0, hi), hi=hi,
                    new_lo=rng.randint(0, new_hi), new_hi=new_hi, T=T,
                    short=rng.choice([0.0, 0.0, rng.random()]))
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    d = rng.choice([16, 64, 64, 72, 96, 128, 128, 128])
    bias = dict(buckets=rng.choice([8, 32, 32, 64, 128]), distance=rng.choice([128, 128, 256, 1024, 2048]),
                bf16=rng.random() < 0.5)
    if op == "decode":
        hi = _log_int(rng, 2, 32768)
        B = _log_int(rng, 1, 32)
        while B > 1 and B * hi * Hkv > 16 * 16896 * 8:
            B = (B + 1) // 2
        return dict(op="decode", B=B, Hq=Hq, Hkv=Hkv, d=d, page=rng.choice([64, 128, 256]),
                    lo=rng.randint(1, hi), hi=hi, **bias)
    causal = rng.random() < 0.6
    B = _log_int(rng, 1, 16)
    hi = _log_int(rng, 2, 4096)
    while B * Hq * hi * hi > 64 * 2048 * 2048:
        B, hi = (B + 1) // 2, hi if B > 1 else hi * 3 // 4
    if rng.random() < 0.5:
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, lo=rng.randint(1, hi), hi=hi,
                    prefix=rng.choice([0, rng.randint(1, 257)]), d=d, causal=causal, **bias)
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, Nq=rng.choice([hi, rng.randint(1, hi)]), Nk=hi, d=d, causal=causal,
                **bias)


def _packed(c):
    return "Nq" not in c


def _spread(lo, hi, n):
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _shapes(c):
    """(queries, keys) of each problem of a forward or backward case."""
    if _packed(c):
        return [(n, n + c["prefix"]) for n in _spread(c["lo"], c["hi"], c["B"])]
    return [(c["Nq"], c["Nk"])] * c["B"]


def _new(c):
    """New tokens of each request of a pages case."""
    n = _spread(c["new_lo"], c["new_hi"], c["B"])
    return n[::2] + n[1::2][::-1]


def work(c):
    if c["op"] == "pages":
        page, old, new = c["page"], _spread(c["lo"], c["hi"], c["B"]), _new(c)
        pages = sum(-(-(o + n) // page) - -(-o // page) for o, n in zip(old, new))
        tokens = c["B"] * c["T"] if c["T"] else sum(new)
        return {"bytes": 12 * tokens + 4 * 4 * pages + 20 * c["B"], "flops": 0}
    row = 2 * c["d"]                                      # bytes of a row of Q, K, V or O
    table = c["buckets"] * c["Hq"] * (2 if c["bf16"] else 4) + 8 * c["distance"]
    if c["op"] == "decode":
        tokens = sum(_spread(c["lo"], c["hi"], c["B"]))
        return {"bytes": 2 * c["Hkv"] * tokens * row + c["B"] * c["Hq"] * (2 * row + 4) + table,
                "flops": 4 * c["Hq"] * c["d"] * tokens}
    shapes = _shapes(c)
    pairs = sum(n * m - (n * (n - 1) // 2 if c["causal"] else 0) for n, m in shapes)
    q, k = (sum(s[i] for s in shapes) for i in (0, 1))
    if c["op"] == "forward":
        return {"bytes": (2 * c["Hq"] * q + 2 * c["Hkv"] * k) * row + 4 * c["Hq"] * q + table,
                "flops": 4 * c["Hq"] * c["d"] * pairs}
    return {"bytes": (4 * c["Hq"] * q + 4 * c["Hkv"] * k) * row + 4 * c["Hq"] * q + 3 * table,
            "flops": 10 * c["Hq"] * c["d"] * pairs}


# ------------------------------------------------------------------ inputs
def _buckets(c):
    """(bucket of each distance from `first` on, first).  Half of a direction's
    buckets hold one distance each, the rest grow geometrically up to
    `distance`; without causal masking each direction has half of them."""
    n = c["buckets"] // (1 if c.get("causal", True) else 2)
    e = n // 2
    s = n - e

    def reaches(r, k):    # distance r is k steps of the geometric part away from e
        return r ** s * e ** k >= c["distance"] ** k * e ** s
    ahead, r, k = [], 0, 0
    while True:
        while r >= e and k + 1 < s and reaches(r, k + 1):
            k += 1
        ahead.append(r if r < e else e + k)
        if ahead[-1] == n - 1:
            break
        r += 1
    back = ahead[::-1]                                     # keys before the query, far to near
    return back + ([] if c.get("causal", True) else [n + b for b in ahead[1:]]), -r


def prepare(c, seed):
    import random
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = random.Random(seed)
    s = dict(c)
    if c["op"] == "pages":
        return _prepare_pages(s, g, rnd, dev)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)

    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    ids, s["first"] = _buckets(c)
    s["ids"] = torch.tensor(ids, dtype=torch.int32, device=dev)
    # a trained table's entries differ by a few units between near and far
    s["table"] = torch.randn(c["buckets"], Hq, generator=g, device=dev) * 1.5
    if c["bf16"]:
        s["table"] = s["table"].to(torch.bfloat16)
    if c["op"] == "decode":
        lengths = _spread(c["lo"], c["hi"], B)
        rnd.shuffle(lengths)
        page = c["page"]
        need = [-(-n // page) for n in lengths]
        perm = torch.randperm(sum(need) + 3, generator=g, device=dev).to(torch.int32)
        first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
        col = torch.arange(max(need), device=dev)
        at = (first[:, None] + col).clamp(max=perm.numel() - 1)
        live = col < torch.tensor(need, device=dev)[:, None]
        s["block_table"] = torch.where(live, perm[at], torch.zeros_like(perm[at])).contiguous()
        s["k_pages"] = randn(perm.numel(), page, Hkv, d)
        s["v_pages"] = randn(perm.numel(), page, Hkv, d)
        s["seqlens"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
        s["q"] = randn(B, Hq, 1, d)
        return s
    if _packed(c):
        shapes = _shapes(c)
        rnd.shuffle(shapes)
        cu_q, cu_k = [0], [0]
        for n, m in shapes:
            cu_q.append(cu_q[-1] + n)
            cu_k.append(cu_k[-1] + m)
        s["q"], s["k"], s["v"] = randn(cu_q[-1], Hq, d), randn(cu_k[-1], Hkv, d), randn(cu_k[-1], Hkv, d)
        s["cu_q"] = torch.tensor(cu_q, dtype=torch.int32, device=dev)
        s["cu_k"] = torch.tensor(cu_k, dtype=torch.int32, device=dev)
        s["max_q"], s["max_k"] = (max(x[i] for x in shapes) for i in (0, 1))
    else:
        s["q"], s["k"], s["v"] = randn(B, Hq, c["Nq"], d), randn(B, Hkv, c["Nk"], d), randn(B, Hkv, c["Nk"], d)
    if c["op"] == "backward":    # a training step holds the forward's output and logsumexp
        s["dout"] = randn(*s["q"].shape)
        s["o"], s["lse"] = _plain_forward(s)
    return s


def _prepare_pages(s, g, rnd, dev):
    B, page = s["B"], s["page"]
    old, new = _spread(s["lo"], s["hi"], B), _new(s)
    rnd.shuffle(old)
    rnd.shuffle(new)
    have = [-(-n // page) for n in old]
    want = [-(-(n + m) // page) - h for n, m, h in zip(old, new, have)]
    free = sum(want) - int(sum(want) * s["short"]) + (5 if s["short"] == 0 else 0)
    blocks = sum(have) + sum(-(-m // page) for m in new) + 5      # (some are not in the pool: lent elsewhere)
    perm = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([0] + have, device=dev).cumsum(0)[:-1]
    col = torch.arange(-(-(s["hi"] + s["new_hi"]) // page) + 1, device=dev)
    at = (first[:, None] + col).clamp(max=blocks - 1)
    live = col < torch.tensor(have, device=dev)[:, None]
    s["block_table"] = torch.where(live, perm[at], torch.full_like(perm[at], -1)).contiguous()
    # the pool: how many pages are free, three words of the library's, then the free pages (the last one goes first)
    s["pool"] = torch.zeros(4 + blocks, dtype=torch.int32, device=dev)
    s["pool"][0] = free
    s["pool"][4:4 + free] = perm[sum(have):sum(have) + free]
    s["seqlens"] = torch.tensor(old, dtype=torch.int32, device=dev)
    s["keep"] = s["seqlens"].clone()
    s["new_lens"] = torch.tensor(new, dtype=torch.int32, device=dev)
    s["total"] = sum(new)
    return s


# --------------------------------------------------------------- one pass
def run(s):
    return {"forward": _forward, "backward": _backward, "decode": _decode, "pages": _pages}[s["op"]](s)


def _forward(s):
    if own:
        import exact_attention_14_gb300 as ea
        if _packed(s):
            return ea.forward_varlen_bias(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], s["max_k"],
                                          s["table"], s["ids"], s["first"], causal=s["causal"])
        return ea.forward_bias(s["q"], s["k"], s["v"], s["table"], s["ids"], s["first"], causal=s["causal"])
    return _plain_forward(s)


def _dense(s):
    """A case as a dense, padded problem in fp32: q, k, v [B, H, N, d], the
    queries' and keys' counts [B], and the places of the live query and key rows."""
    q, k, v = s["q"], s["k"], s["v"]
    if not _packed(s):
        B = s["B"]
        nq, nk = (torch.full((B,), x.shape[2], device=q.device) for x in (q, k))
        return q.float(), k.float(), v.float(), nq, nk, None, None
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    nq, nk = cu_q.diff(), cu_k.diff()
    at_q, live_q = _padded(cu_q, s["max_q"], q.shape[0])
    at_k, live_k = _padded(cu_k, s["max_k"], k.shape[0])
    return (q[at_q].transpose(1, 2).float(), k[at_k].transpose(1, 2).float(), v[at_k].transpose(1, 2).float(),
            nq, nk, live_q, live_k)


def _padded(cu, n, total):
    i = torch.arange(n, device=cu.device)
    return (cu[:-1, None] + i).clamp(max=total - 1), i < cu.diff()[:, None]


def _scores(s, q, k, nq, nk):
    """scale q k^T + bias with -inf where a query does not see a key: [B, Hq, Nq, Nk] fp32."""
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    x = (q.reshape(B, Hkv, -1, d) @ k.transpose(2, 3)).view(B, Hq, Nq, Nk).mul_(d ** -0.5)
    i = torch.arange(Nq, device=q.device)[:, None]
    j = torch.arange(Nk, device=q.device)
    offset = (nk - nq) if _packed(s) else (nk - nq)[:1]
    r = j - i - offset[:, None, None]                                  # [B or 1, Nq, Nk]
    x += s["table"].float().t()[:, s["ids"].long()[(r - s["first"]).clamp(0, s["ids"].numel() - 1)]].transpose(0, 1)
    out = j >= nk[:, None, None]
    if s["causal"]:
        out = out | (r > 0)
    return x.masked_fill_(out[:, None], -math.inf)


def _plain_forward(s):
    q, k, v, nq, nk, live_q, _ = _dense(s)
    B, Hq, Nq, d = q.shape
    p = _scores(s, q, k, nq, nk)
    m = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p = p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, k.shape[1], -1, k.shape[2]) @ v).view(B, Hq, Nq, d) / total.clamp(min=1e-30)
    lse = (m + total.log()).squeeze(-1)
    o = o.to(torch.bfloat16)
    if _packed(s):
        return o.transpose(1, 2)[live_q], lse.transpose(0, 1)[:, live_q].contiguous()
    return o, lse


def _backward(s):
    if own:
        import exact_attention_14_gb300 as ea
        if _packed(s):
            return ea.backward_varlen_bias(s["q"], s["k"], s["v"], s["o"], s["dout"], s["lse"], s["cu_q"],
                                           s["cu_k"], s["max_q"], s["max_k"], s["table"], s["ids"], s["first"],
                                           causal=s["causal"])
        return ea.backward_bias(s["q"], s["k"], s["v"], s["o"], s["dout"], s["lse"], s["table"], s["ids"],
                                s["first"], causal=s["causal"])
    q, k, v, nq, nk, live_q, live_k = _dense(s)
    B, Hq, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if _packed(s):    # rows past a sequence's last query have no gradient
        at, _ = _padded(s["cu_q"].long(), Nq, s["q"].shape[0])
        dout = (s["dout"][at].float() * live_q[..., None, None]).transpose(1, 2)
        delta = (dout * s["o"][at].transpose(1, 2).float()).sum(-1, keepdim=True)
        lse = s["lse"][:, at].transpose(0, 1)[..., None]
    else:
        dout = s["dout"].float()
        delta = (dout * s["o"].float()).sum(-1, keepdim=True)
        lse = s["lse"][..., None]
    p = _scores(s, q, k, nq, nk).sub_(lse).exp_()
    if _packed(s):
        p *= live_q[:, None, :, None]
    rows = (B, Hkv, -1, d)
    cols = (B, Hkv, -1, Nk)
    dv = p.view(cols).transpose(2, 3) @ dout.reshape(rows)
    ds = (dout.reshape(rows) @ v.transpose(2, 3)).view(p.shape).sub_(delta).mul_(p)
    del p
    dq = ((ds.view(cols) @ k) * d ** -0.5).view(B, Hq, Nq, d).to(torch.bfloat16)
    dk = ((ds.view(cols).transpose(2, 3) @ q.reshape(rows)) * d ** -0.5).to(torch.bfloat16)
    dv = dv.to(torch.bfloat16)
    # every diagonal of dS: with the rows upside down and each one column further, a diagonal is a column
    skew = torch.nn.functional.pad(ds.flip(2), (0, Nq)).flatten(2)[..., :-Nq].view(B, Hq, Nq, Nk + Nq - 1)
    along = skew.sum(2, dtype=torch.float64)                           # [B, Hq, distances]
    r = torch.arange(1 - Nq, Nk, device=q.device) - (nk - nq)[:, None]
    at = s["ids"].long()[(r - s["first"]).clamp(0, s["ids"].numel() - 1)].reshape(-1)
    dtable = torch.zeros(s["table"].shape, dtype=torch.float64, device=q.device)
    dtable.index_add_(0, at, along.transpose(1, 2).reshape(-1, Hq))
    if _packed(s):
        dq, dk, dv = dq.transpose(1, 2)[live_q], dk.transpose(1, 2)[live_k], dv.transpose(1, 2)[live_k]
    return dq, dk, dv, dtable.float()


def _decode(s):
    if own:
        import exact_attention_14_gb300 as ea
        return ea.decode_paged_bias(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seqlens"], s["table"],
                                    s["ids"], s["first"])
    B, Hq, _, d = s["q"].shape
    Hkv = s["Hkv"]
    table = s["block_table"].long()
    n = table.shape[1] * s["page"]
    k, v = (x[table].reshape(B, n, Hkv, d).transpose(1, 2).float() for x in (s["k_pages"], s["v_pages"]))
    L = s["seqlens"].long()
    j = torch.arange(n, device=L.device)
    x = (s["q"].float().view(B, Hkv, -1, d) @ k.transpose(2, 3)).view(B, Hq, n) * d ** -0.5
    r = j - (L[:, None] - 1)
    x = x + s["table"].float()[s["ids"].long()[(r - s["first"]).clamp(0, s["ids"].numel() - 1)]].transpose(1, 2)
    x = x.masked_fill((r > 0)[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, n) @ v).view(B, Hq, d) / total
    return o.view(B, Hq, 1, d).to(torch.bfloat16), m + total.log()


def _pages(s):
    """A step's new tokens get their pages and slots; the step's requests then give them back, so that the
    state is what it was."""
    if own:
        import exact_attention_14_gb300 as ea
        got = ea.pages_extend(s["pool"], s["block_table"], s["seqlens"], s["new_lens"], s["page"],
                              **({"width": s["T"]} if s["T"] else {"total": s["total"]}))
        ea.pages_trim(s["pool"], s["block_table"], s["seqlens"], s["keep"], s["page"])
        return (*got, s["seqlens"], s["block_table"], s["pool"])
    page, pool, table = s["page"], s["pool"], s["block_table"]
    B, width = table.shape
    old, new, count = s["seqlens"].long(), s["new_lens"].long(), pool[0].long()
    have = (old + page - 1) // page
    need = (old + new + page - 1) // page - have
    upto = need.cumsum(0)
    given = (need == 0) | (upto <= count)
    col = torch.arange(width, device=old.device)
    nth = (upto - need)[:, None] + col - have[:, None]                # which of the step's pages
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None]) & given[:, None]
    table.copy_(torch.where(fresh, pool[(4 + count - 1 - nth).clamp(4, pool.numel() - 1)], table))
    granted = torch.where(given, new, torch.zeros_like(new))
    if s["T"]:
        t = torch.arange(s["T"], device=old.device).expand(B, -1)
        b = torch.arange(B, device=old.device)[:, None].expand(-1, s["T"])
        cu = ()
    else:
        ends = new.cumsum(0)
        n = torch.arange(s["total"], device=old.device)
        b = torch.searchsorted(ends, n, right=True)
        t = n - (ends - new)[b]
        cu = (torch.nn.functional.pad(ends, (1, 0)).to(torch.int32),)
    pos = old[b] + t
    asked = t < new[b]
    live = t < granted[b]
    at = table.long()[b, (pos // page).clamp(max=width - 1)]
    slots = torch.where(live, at * page + pos % page, torch.full_like(pos, -1))
    positions = torch.where(asked, pos, torch.zeros_like(pos)).to(torch.int32)
    s["seqlens"].add_(granted.to(torch.int32))
    pool[0] -= torch.where(given, need, torch.zeros_like(need)).sum().to(torch.int32)
    # and back: the pages past the kept tokens, the last one deepest
    now, keep, count = s["seqlens"].long(), s["keep"].long(), pool[0].long()
    keep = torch.minimum(keep.clamp(min=0), now)
    kept = (keep + page - 1) // page
    back = (now + page - 1) // page - kept
    upto = back.cumsum(0)
    nth = (upto - back)[:, None] + col - kept[:, None]
    gone = (col >= kept[:, None]) & (col < (kept + back)[:, None])
    pool.scatter_(0, torch.where(gone, 4 + count + upto[-1] - 1 - nth, torch.ones_like(nth)).reshape(-1),
                  torch.where(gone, table, torch.zeros_like(table)).reshape(-1))
    pool[0] += upto[-1].to(torch.int32)
    s["seqlens"].copy_(keep)
    return (slots, positions, *cu, granted.to(torch.int32), s["seqlens"], table, pool)


# ------------------------------------------------------------------ 64 bits
def exact(c, seed):
    if c["op"] == "pages":
        return None
    s = prepare(c, seed)
    dev = s["q"].device
    Hq, d = c["Hq"], c["d"]
    G = Hq // c["Hkv"]
    ids, table = s["ids"].cpu().long(), s["table"].double()

    def bias(n, m, h):    # [n, m] of head h, the last query at the last key
        near = torch.arange(m, device=dev) - torch.arange(n, device=dev)[:, None] - (m - n)
        return table[ids.to(dev), h][torch.clamp(near - s["first"], 0, len(ids) - 1)]

    if c["op"] == "decode":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
        lse = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device=dev)
        for b, L in enumerate(s["seqlens"].tolist()):
            pages = s["block_table"][b, :-(-L // c["page"])].long()
            k = s["k_pages"][pages].flatten(0, 1)[:L].double()
            v = s["v_pages"][pages].flatten(0, 1)[:L].double()
            for h in range(Hq):
                x = k[:, h // G] @ s["q"][b, h, 0].double() / math.sqrt(d) + bias(1, L, h)[0]
                lse[b, h, 0] = torch.logsumexp(x, 0)
                o[b, h, 0] = torch.exp(x - lse[b, h, 0]) @ v[:, h // G]
        return o, lse

    packed = _packed(c)
    cq = s["cu_q"].tolist() if packed else None
    ck = s["cu_k"].tolist() if packed else None

    def part(x, cu, b, h):    # problem b, head h of a tensor, as [rows, d]
        return x[cu[b]:cu[b + 1], h] if packed else x[b, h]

    def stat(x, b, h):
        return x[h, cq[b]:cq[b + 1]] if packed else x[b, h]

    def zeros(x):
        return torch.zeros(x.shape, dtype=torch.float64, device=dev)

    outs = [zeros(s["q"]), torch.zeros((Hq, s["q"].shape[0]) if packed else s["q"].shape[:3], dtype=torch.float64,
                                       device=dev)]
    if c["op"] == "backward":
        outs = [zeros(s["q"]), zeros(s["k"]), zeros(s["v"]), zeros(s["table"])]
    for b in range(c["B"]):
        for h in range(Hq):
            q, k, v = (part(x, cu, b, i).double() for x, cu, i in ((s["q"], cq, h), (s["k"], ck, h // G),
                                                                   (s["v"], ck, h // G)))
            n, m = q.shape[0], k.shape[0]
            x = torch.addmm(bias(n, m, h), q, k.T, alpha=1 / math.sqrt(d))
            if c["causal"]:
                x.masked_fill_(torch.ones(n, m, dtype=torch.bool, device=dev).triu(m - n + 1), -math.inf)
            if c["op"] == "forward":
                z = torch.logsumexp(x, 1)
                stat(outs[1], b, h).copy_(z)
                part(outs[0], cq, b, h).copy_(torch.exp(x - torch.nan_to_num(z, neginf=0.0)[:, None]) @ v)
                continue
            do = part(s["dout"], cq, b, h).double()
            p = torch.exp(x - stat(s["lse"], b, h).double()[:, None])
            part(outs[2], ck, b, h // G).add_(p.T @ do)
            p *= do @ v.T - (do * part(s["o"], cq, b, h).double()).sum(1)[:, None]
            part(outs[0], cq, b, h).copy_(p @ k / math.sqrt(d))
            part(outs[1], ck, b, h // G).add_(p.T @ q / math.sqrt(d))
            # keys reversed, rows read back at one column less than they were laid out: a column is a distance
            flip = torch.zeros(n, n + m, dtype=torch.float64, device=dev)
            flip[:, :m] = p.flip(1)
            sums = flip.view(-1)[:n * (n + m - 1)].view(n, n + m - 1).sum(0)   # column (m - 1 - j) + i
            r = (m - 1 - torch.arange(n + m - 1, device=dev)) - (m - n)
            at = ids.to(dev)[torch.clamp(r - s["first"], 0, len(ids) - 1)]
            outs[3][:, h] += torch.zeros(table.shape[0], dtype=torch.float64, device=dev).index_add_(0, at, sums)
    return tuple(outs)
