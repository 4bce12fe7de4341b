"""The positions, cache and tree-attention operators as they are measured.

Four kinds of case, told apart by ``op``:

  rope    rotary positions on Q and K (``inverse`` is the gradient)
  write   keys and values written into a paged cache, bf16 or E4M3
  read    a paged cache read back into packed keys and values
  tree    attention of the drafted tokens of each sequence over a paged cache

With ``own`` false, ``run`` computes an operator with elementary torch
operations in 32 bits (angles in 64); with ``own`` true it calls the library.
``exact`` computes the same in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY_AMAX = 2.0 ** -100      # a smaller row's scale is the one of this maximum


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's positions: 16 sequences, one token each, far into their contexts
        dict(name="rope_step", op="rope", B=16, N=1, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             scaling="none", factor=1.0, far=32768, token_major=False, inverse=False, f32=False),
        # prefill of 8 x 4096 tokens straight from a projection's token-major rows, long-context scaling
        dict(name="rope_prefill", op="rope", B=8, N=4096, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, scaling="parts", factor=8.0, far=131072, token_major=True,
             inverse=False, f32=False),
        # the gradient of a partly rotated, interleaved head; odd length; fp32 gradients
        dict(name="rope_grad_odd", op="rope", B=3, N=1531, Hq=12, Hkv=4, d=96, rot=40, interleaved=True,
             scaling="ntk", factor=4.0, far=0, token_major=False, inverse=True, f32=True),
        # one decode step's keys and values into an 8-bit cache
        dict(name="write_step_e4m3", op="write", B=16, N=1, Hkv=8, d=128, page=64, e4m3=True, pad=0),
        # a prefill's keys and values (8 x 4096 tokens) into an 8-bit cache, some tokens padding
        dict(name="write_prefill_e4m3", op="write", B=8, N=4096, Hkv=8, d=128, page=64, e4m3=True,
             pad=7),
        # 16-key pages read back at odd lengths and d = 96 for a chunk of a prompt
        dict(name="read_odd_bf16", op="read", B=5, Hkv=4, d=96, page=16, e4m3=False, lo=1, hi=2999),
        # the decode workload's whole 8-bit cache read back
        dict(name="read_long_e4m3", op="read", B=16, Hkv=8, d=128, page=64, e4m3=True, lo=1024,
             hi=32768),
        # a few drafted tokens over short, odd contexts: latency
        dict(name="tree_small_bf16", op="tree", B=3, Hq=8, Hkv=2, T=7, d=96, page=16, e4m3=False, lo=40,
             hi=777, chain=False, ragged=True),
        # the decode workload, one token each, over an 8-bit cache
        dict(name="tree_decode_e4m3", op="tree", B=16, Hq=32, Hkv=8, T=1, d=128, page=64, e4m3=True,
             lo=1024, hi=32768, chain=True, ragged=False),
        # the decode workload with 16 drafted tokens in a tree
        dict(name="tree_16_bf16", op="tree", B=16, Hq=32, Hkv=8, T=16, d=128, page=64, e4m3=False,
             lo=1024, hi=32768, chain=False, ragged=True),
        # 64 drafted tokens over the 8-bit cache
        dict(name="tree_64_e4m3", op="tree", B=16, Hq=32, Hkv=8, T=64, d=128, page=64, e4m3=True,
             lo=1024, hi=32768, chain=False, ragged=False),
        # 64 drafted tokens over the bf16 cache: the largest
        dict(name="tree_64_bf16", op="tree", B=16, Hq=32, Hkv=8, T=64, d=128, page=64, e4m3=False,
             lo=1024, hi=32768, chain=False, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "tree", "tree"])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 192, 256])
        N = _log_int(rng, 1, 8192)
        B = max(1, min(_log_int(rng, 1, 64), 40000 // N))
        return dict(op="rope", B=B, N=N, Hq=Hkv * rng.choice([1, 2, 4, 8]), Hkv=Hkv, d=d,
                    rot=2 * rng.randint(1, d // 2) if rng.random() < 0.5 else d,
                    interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "parts"]),
                    factor=rng.choice([2.0, 4.0, 8.0, 32.0]), far=_log_int(rng, 1, 1 << 20),
                    token_major=rng.random() < 0.5, inverse=rng.random() < 0.5,
                    f32=rng.random() < 0.3)
    e4m3 = rng.random() < 0.5
    d = rng.choice([32, 64, 80, 96, 128, 128, 192, 256] if e4m3 else [40, 64, 72, 96, 128, 128, 200, 256])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "write":
        N = _log_int(rng, 1, 8192)
        return dict(op="write", B=max(1, min(_log_int(rng, 1, 64), 40000 // N)), N=N, Hkv=Hkv, d=d,
                    page=page, e4m3=e4m3, pad=rng.choice([0, 3, 11]) if N > 1 else 0)
    B = _log_int(rng, 1, 32)
    hi = _log_int(rng, 2, 32768)
    lo = rng.randint(1, hi)
    if op == "read":
        while B * (lo + hi) * Hkv * d > 16 * 33792 * 8 * 128:
            hi = (hi + 1) // 2
            lo = min(lo, hi)
        return dict(op="read", B=B, Hkv=Hkv, d=d, page=page, e4m3=e4m3, lo=lo, hi=hi)
    T = _log_int(rng, 1, 64)
    G = rng.choice([1, 2, 4, 8])
    hi = max(hi, T)
    lo = max(lo, T)
    while B > 1 and B * (lo + hi) * Hkv * d * max(T * G, 256) > 16 * 33792 * 8 * 128 * 256:
        B = (B + 1) // 2
    return dict(op="tree", B=B, Hq=Hkv * G, Hkv=Hkv, T=T, d=d, page=page, e4m3=e4m3, lo=lo, hi=max(lo, hi),
                chain=rng.random() < 0.3, ragged=rng.random() < 0.5)


def _lengths(c):
    """The cached lengths of a case: evenly spread over [lo, hi]."""
    B = c["B"]
    return [c["hi"] if B == 1 else c["lo"] + (c["hi"] - c["lo"]) * b // (B - 1) for b in range(B)]


def work(c):
    if c["op"] == "rope":
        rows = c["B"] * c["N"] * (c["Hq"] + c["Hkv"])
        size = 4 if c["f32"] else 2
        return {"bytes": 2 * rows * c["d"] * size + 4 * c["B"] * c["N"] + 4 * c["rot"],
                "flops": 3 * rows * c["rot"]}
    row = c["d"] * (1 if c["e4m3"] else 2) + (4 if c["e4m3"] else 0)    # a cached K or V row
    if c["op"] == "write":
        rows = 2 * c["Hkv"] * (c["B"] * c["N"] - _padding(c))
        return {"bytes": rows * (2 * c["d"] + row) + 8 * c["B"] * c["N"], "flops": 2 * rows * c["d"]}
    tokens = sum(_lengths(c))
    if c["op"] == "read":
        rows = 2 * c["Hkv"] * tokens
        return {"bytes": rows * (row + 2 * c["d"]), "flops": rows * c["d"]}
    drafted = sum(_drafted(c))
    return {"bytes": 2 * c["Hkv"] * tokens * row + drafted * c["Hq"] * (2 * c["d"] + 2 * c["d"] + 4),
            "flops": sum(4 * n * c["Hq"] * c["d"] * L for n, L in zip(_drafted(c), _lengths(c)))}


def _padding(c):
    """Tokens of a write case that are padding: every pad-th one."""
    return -(-c["B"] * c["N"] // c["pad"]) if c["pad"] else 0


def _drafted(c):
    """Drafted tokens of each sequence of a tree case."""
    return [max(1, c["T"] - (b * 5) % c["T"]) if c["ragged"] else c["T"] for b in range(c["B"])]


# ------------------------------------------------------------------ inputs
def _frequencies(c):
    """Radians per position of each rotated pair (fp64), and the magnitude factor."""
    rot, base, s = c["rot"], 10000.0, c["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    if c["scaling"] == "ntk" and rot > 2:
        base = base * s ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] != "parts":
        return f, 1.0

    def at(turns):    # the (fractional) pair that turns this often over 4096 positions
        return rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(base))
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot // 2 - 1)
    keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f / s * (1 - keep) + f * keep, 0.1 * math.log(s) + 1.0


def _table(g, lengths, page, width, dev):
    """Pages of every sequence, scattered over the cache: the block table, and the page count."""
    need = [-(-n // page) for n in lengths]
    total = sum(need) + 3
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([0] + need, device=dev).cumsum(0)[:-1]
    col = torch.arange(width, device=dev)
    at = (first[:, None] + col[None, :]).clamp(max=total - 1)
    live = col[None, :] < torch.tensor(need, device=dev)[:, None]
    return torch.where(live, perm[at], torch.zeros_like(perm[at])).contiguous(), total


def _pages(g, blocks, c, dev):
    """One cache of K (or V): pages, and for E4M3 the descales [blocks, Hkv, page]."""
    x = torch.randn(blocks, c["page"], c["Hkv"], c["d"], generator=g, device=dev, dtype=torch.bfloat16)
    if not c["e4m3"]:
        return x, None
    amax = x.abs().amax(-1)
    scale = E4M3_MAX / amax.float()
    codes = (x.float() * scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    # a cache's rows differ in size: some tokens' keys and values are larger than others'
    size = torch.rand(blocks, c["Hkv"], c["page"], generator=g, device=dev) * 1.5 + 0.25
    return codes, ((amax.float() / E4M3_MAX).transpose(1, 2) * size).contiguous()


def _words(mask):
    """bool [B, T, U] -> int64 [B, T, ceil(U / 64)] with bit u % 64 of word u // 64 for u."""
    B, T, U = mask.shape
    W = -(-U // 64)
    m = torch.zeros(B, T, W * 64, dtype=torch.int64)
    m[..., :U] = mask
    return (m.reshape(B, T, W, 64) << torch.arange(64)).sum(-1)


def prepare(c, seed):
    import random
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = random.Random(seed)
    s = dict(c)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    if c["op"] == "rope":
        dt = torch.float32 if c["f32"] else torch.bfloat16
        B, N = c["B"], c["N"]
        if c["token_major"]:    # a projection's output: all heads of a token together
            both = randn(B, N, c["Hq"] + c["Hkv"], c["d"], dtype=dt)
            s["q"] = both[:, :, :c["Hq"]].transpose(1, 2)
            s["k"] = both[:, :, c["Hq"]:].transpose(1, 2)
        else:
            s["q"] = randn(B, c["Hq"], N, c["d"], dtype=dt)
            s["k"] = randn(B, c["Hkv"], N, c["d"], dtype=dt)
        start = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device=dev)
        s["positions"] = (start + torch.arange(N, device=dev)).to(torch.int32)
        f, s["magnitude"] = _frequencies(c)
        s["inv_freq"] = f.to(dev)
        return s
    if c["op"] == "write":
        B, N, page = c["B"], c["N"], c["page"]
        s["k"] = randn(B, c["Hkv"], N, c["d"])
        s["v"] = randn(B, N, c["Hkv"], c["d"]).transpose(1, 2)
        blocks = -(-B * N // page) + 2
        slots = torch.randperm(blocks * page, generator=g, device=dev)[:B * N].reshape(B, N)
        if N > 1:    # a sequence's tokens lie page by page
            order = torch.randperm(blocks, generator=g, device=dev)
            t = torch.arange(B * N, device=dev)
            slots = (order[t // page] * page + t % page).reshape(B, N)
        if c["pad"]:
            slots.view(-1)[::c["pad"]] = -1
        s["slots"] = slots.contiguous()
        kind = torch.uint8 if c["e4m3"] else torch.bfloat16
        s["k_pages"] = torch.zeros(blocks, page, c["Hkv"], c["d"], dtype=kind, device=dev)
        s["v_pages"] = torch.zeros_like(s["k_pages"])
        s["k_descale"] = s["v_descale"] = None
        if c["e4m3"]:
            s["k_descale"] = torch.ones(blocks, c["Hkv"], page, device=dev)
            s["v_descale"] = torch.ones(blocks, c["Hkv"], page, device=dev)
        return s
    lengths = _lengths(c)
    if c["op"] == "read":
        rnd.shuffle(lengths)
    width = -(-max(lengths) // c["page"])
    s["block_table"], blocks = _table(g, lengths, c["page"], width, dev)
    s["k_pages"], s["k_descale"] = _pages(g, blocks, c, dev)
    s["v_pages"], s["v_descale"] = _pages(g, blocks, c, dev)
    if c["op"] == "read":
        s["total"] = sum(lengths)
        s["cu_seqlens"] = torch.tensor([0] + lengths, device=dev).cumsum(0).to(torch.int32)
        return s
    s["seqlens"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["q"] = randn(c["B"], c["Hq"], c["T"], c["d"])
    s["tree_mask"] = None
    if not c["chain"]:    # random trees: drafted token t sees itself and its ancestors
        mask = torch.zeros(c["B"], c["T"], c["T"], dtype=torch.bool)
        for b in range(c["B"]):
            for t in range(c["T"]):
                parent = rnd.randrange(-1, t)
                if parent >= 0:
                    mask[b, t] = mask[b, parent]
                mask[b, t, t] = True
        s["tree_mask"] = _words(mask).to(dev)
    s["q_lens"] = torch.tensor(_drafted(c), dtype=torch.int32, device=dev) if c["ragged"] else None
    return s


# --------------------------------------------------------------- one pass
def run(s):
    return {"rope": _rope, "write": _write, "read": _read, "tree": _tree}[s["op"]](s)


def _rope(s):
    if own:
        import exact_attention_14_gb300 as ea
        return (ea.rope_backward if s["inverse"] else ea.rope)(
            s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=s["interleaved"],
            magnitude=s["magnitude"])
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"]
    if s["inverse"]:
        angle = -angle
    cos, sin = angle.cos().float() * s["magnitude"], angle.sin().float() * s["magnitude"]
    return _turned(s["q"], cos, sin, s), _turned(s["k"], cos, sin, s)


def _turned(x, cos, sin, s):
    rot = s["rot"]
    x32 = x.float()
    y = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., lo] = x32[..., lo] * cos - x32[..., hi] * sin
    y[..., hi] = x32[..., lo] * sin + x32[..., hi] * cos
    y[..., rot:] = x32[..., rot:]
    return y.to(x.dtype)


def _write(s):
    if own:
        import exact_attention_14_gb300 as ea
        ea.attn_cache_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"], s["k_descale"],
                            s["v_descale"])
    else:
        _write_one(s["k"], s["k_pages"], s["k_descale"], s["slots"].reshape(-1), s)
        _write_one(s["v"], s["v_pages"], s["v_descale"], s["slots"].reshape(-1), s)
    if not s["e4m3"]:
        return s["k_pages"], s["v_pages"]
    return (s["k_pages"].view(torch.float8_e4m3fn), s["v_pages"].view(torch.float8_e4m3fn),
            s["k_descale"], s["v_descale"])


def _write_one(x, pages, descale, slots, s):
    rows = x.transpose(1, 2).reshape(-1, s["Hkv"], s["d"])
    at = slots
    if s["pad"]:    # a padding token repeats the first live one
        live = slots >= 0
        src = torch.where(live, torch.arange(slots.numel(), device=slots.device), live.int().argmax())
        at, rows = slots[src], rows[src]
    if s["e4m3"]:
        rows = rows.float()
        amax = rows.abs().amax(-1)
        scaled = amax.clamp(min=TINY_AMAX)
        one = torch.where(amax > 0, scaled / E4M3_MAX, torch.ones_like(amax))
        # (a number over a tensor would be a reciprocal and a product: two roundings)
        scale = torch.full_like(scaled, E4M3_MAX) / scaled
        rows = rows * torch.where(amax > 0, scale, torch.ones_like(amax))[..., None]
        rows = rows.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        descale[at // s["page"], :, at % s["page"]] = one
    pages.view(-1, s["Hkv"], s["d"])[at] = rows


def _read(s):
    if own:
        import exact_attention_14_gb300 as ea
        return ea.cache_read(s["k_pages"], s["v_pages"], s["block_table"], s["cu_seqlens"], s["total"],
                             s["k_descale"], s["v_descale"])
    cu = s["cu_seqlens"].long()
    token = torch.arange(s["total"], device=cu.device)
    b = torch.searchsorted(cu, token, right=True) - 1
    pos = token - cu[b]
    at = s["block_table"].long()[b, pos // s["page"]] * s["page"] + pos % s["page"]
    return tuple(_rows(pages, descale, at, s) for pages, descale in
                 ((s["k_pages"], s["k_descale"]), (s["v_pages"], s["v_descale"])))


def _rows(pages, descale, at, s):
    rows = pages.reshape(-1, s["Hkv"], s["d"])[at]
    if s["e4m3"]:
        rows = rows.view(torch.float8_e4m3fn).float() * descale[at // s["page"], :, at % s["page"]][..., None]
    return rows.to(torch.bfloat16)


def _allowed(s, n, L, lens):
    """bool [B, T, n]: the keys that each drafted token attends; rows past a sequence's drafted tokens none."""
    dev = L.device
    T = s["T"]
    key = torch.arange(n, device=dev)[None, None, :]
    first = (L - lens)[:, None, None]
    u = key - first                                    # drafted token that a key belongs to
    row = torch.arange(T, device=dev)[None, :, None]
    if s["tree_mask"] is None:
        seen = u <= row
    else:
        word = u.clamp(0, T - 1)
        words = torch.gather(s["tree_mask"], 2, (word // 64).expand(-1, T, -1))
        seen = ((words >> (word % 64)) & 1).bool()
    return ((key < first) | ((u >= 0) & (u < lens[:, None, None]) & seen)) & (row < lens[:, None, None])


def _tree(s):
    if own:
        import exact_attention_14_gb300 as ea
        return ea.decode_tree(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seqlens"],
                              s["tree_mask"], s["q_lens"], s["k_descale"], s["v_descale"])
    B, Hq, T, d = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]
    L = s["seqlens"].long()
    lens = torch.full_like(L, T) if s["q_lens"] is None else s["q_lens"].long()
    n = s["block_table"].shape[1] * page
    table = s["block_table"].long()

    def keys(pages, descale):
        x = pages[table]                                           # [B, blocks, page, Hkv, d]
        if s["e4m3"]:
            x = x.view(torch.float8_e4m3fn).float() * descale[table].transpose(2, 3)[..., None]
        return x.float().reshape(B, n, Hkv, d).transpose(1, 2)     # [B, Hkv, n, d]

    q = s["q"].float().reshape(B, Hkv, -1, d)                      # rows (g, t)
    p = q @ keys(s["k_pages"], s["k_descale"]).transpose(2, 3) * d ** -0.5
    p = p.view(B, Hkv, -1, T, n).masked_fill_(~_allowed(s, n, L, lens)[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    p = (p - m.clamp(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Hkv, -1, n) @ keys(s["v_pages"], s["v_descale"])).view(B, Hkv, -1, T, d)
    out = out / total.clamp(min=1e-30)
    lse = (m + total.log()).squeeze(-1)
    return out.reshape(B, Hq, T, d).to(torch.bfloat16), lse.reshape(B, Hq, T)


# ------------------------------------------------------------------ 64 bits
def _e4m3_64(x):
    """x (fp64, |x| <= 448) rounded to the nearest E4M3 value, ties to even."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -60)))
    e = torch.where(torch.exp2(e) > a, e - 1, e)
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, e).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        angle = s["positions"].double().unsqueeze(1).unsqueeze(-1) * s["inv_freq"]
        z = torch.polar(torch.full_like(angle, s["magnitude"]), -angle if c["inverse"] else angle)
        rot = c["rot"]

        def turn(x):
            y = x.double().clone()
            pair = y[..., :rot].unflatten(-1, (-1, 2) if c["interleaved"] else (2, -1))
            pair = pair if c["interleaved"] else pair.transpose(-1, -2)
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            y[..., :rot] = (w if c["interleaved"] else w.transpose(-1, -2)).flatten(-2)
            return y
        return turn(s["q"]), turn(s["k"])
    if c["op"] == "write":
        flat = s["slots"].flatten()
        tok = torch.nonzero(flat >= 0).squeeze(1)
        where = flat[tok]
        got = []
        for x, pages in ((s["k"], s["k_pages"]), (s["v"], s["v_pages"])):
            rows = x.double().permute(0, 2, 1, 3).flatten(0, 1).index_select(0, tok)
            store = torch.zeros(pages.shape, dtype=torch.float64, device=x.device)
            scales = torch.ones(pages.shape[0], c["page"], c["Hkv"], dtype=torch.float64, device=x.device)
            if c["e4m3"]:
                top = rows.abs().max(-1).values
                part = torch.where(top > 0, top, torch.ones_like(top)).unsqueeze(-1)
                rows = _e4m3_64(rows * E4M3_MAX / part)
                scales.flatten(0, 1).index_copy_(0, where, torch.where(top > 0, top / E4M3_MAX,
                                                                       torch.ones_like(top)))
            store.flatten(0, 1).index_copy_(0, where, rows)
            got.append((store, scales.permute(0, 2, 1)))
        values = [x[0] for x in got]
        return tuple(values + [x[1] for x in got]) if c["e4m3"] else tuple(values)

    def cached(pages, descale):
        if c["e4m3"]:
            return pages.view(torch.float8_e4m3fn).double() * descale.double().permute(0, 2, 1).unsqueeze(-1)
        return pages.double()
    if c["op"] == "read":
        cu = s["cu_seqlens"].tolist()
        outs = []
        for pages, descale in ((s["k_pages"], s["k_descale"]), (s["v_pages"], s["v_descale"])):
            parts = []
            for b in range(c["B"]):
                n = cu[b + 1] - cu[b]
                ids = s["block_table"][b, :-(-n // c["page"])].long()
                x = cached(pages[ids], None if descale is None else descale[ids])
                parts.append(x.flatten(0, 1)[:n])
            outs.append(torch.cat(parts))
        return tuple(outs)
    B, Hq, T, d = s["q"].shape
    G = Hq // c["Hkv"]
    o = torch.zeros(B, Hq, T, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        L = int(s["seqlens"][b])
        n = T if s["q_lens"] is None else int(s["q_lens"][b])
        ids = s["block_table"][b, :-(-L // c["page"])].long()
        k = cached(s["k_pages"][ids], None if s["k_descale"] is None else s["k_descale"][ids]).flatten(0, 1)[:L]
        v = cached(s["v_pages"][ids], None if s["v_descale"] is None else s["v_descale"][ids]).flatten(0, 1)[:L]
        see = torch.tril(torch.ones(n, n, dtype=torch.bool, device=k.device))
        if s["tree_mask"] is not None:
            bits = torch.arange(n, device=k.device)
            see = ((s["tree_mask"][b, :n][:, bits // 64] >> (bits % 64)) & 1).bool()
        for h in range(c["Hkv"]):
            q = s["q"][b, h * G:(h + 1) * G, :n].double()
            x = q @ k[:, h].T / math.sqrt(d)
            x[..., L - n:] = x[..., L - n:].masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, -1)
            lse[b, h * G:(h + 1) * G, :n] = z
            o[b, h * G:(h + 1) * G, :n] = torch.nan_to_num(torch.exp(x - z.unsqueeze(-1))) @ v[:, h]
    return o, lse
