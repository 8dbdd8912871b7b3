"""Cases of the serving operators around a paged 4-bit KV cache: page bookkeeping, per-head norm with rotation,
writing and reading the cache, and decode over it.  Every case has a plain torch form beside the framework's call.

The cache is a pool of bytes [num_pages, Hkv, page_size / 16, tile_bytes].  A tile holds 16 keys of one head: the K
codes as [D / 64][16 keys][32 bytes], the V codes alike, then K's and V's (scale, minimum) pairs as fp16
[16 keys][D / 64][2].  Byte j of a code row holds dims 2 j (low half) and 2 j + 1 of its group of 64, and a code u
stands for scale * u + minimum.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F16_MAX = 65504.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One decode step of eight running requests (the repository's GQA decode lengths): a page now and then.
        {"name": "pages_decode_8", "kind": "pages", "B": 8, "page": 16, "lo": 512, "hi": 4096, "nlo": 1, "nhi": 1,
         "lens": 1},
        # Sixteen prompts of 256 to 8192 tokens arrive at once and are released after scoring: every token's slot.
        {"name": "pages_prompts_16", "kind": "pages", "B": 16, "page": 16, "lo": 0, "hi": 0, "nlo": 256, "nhi": 8192,
         "lens": 2},
        # q and k of one decode step, eight tokens out of a fused projection: latency.
        {"name": "norm_decode_8", "kind": "norm", "T": 8, "Hq": 32, "Hkv": 8, "D": 128, "style": "half", "pad": 0,
         "maxpos": 4096},
        # The same for the prompts of a ragged prefill batch: bandwidth.
        {"name": "norm_prompts_64k", "kind": "norm", "T": 65536, "Hq": 32, "Hkv": 8, "D": 128, "style": "half",
         "pad": 0, "maxpos": 8192},
        # A model of smaller heads with interleaved pairs, an odd number of tokens in a batch padded for a graph.
        {"name": "norm_d64_padded", "kind": "norm", "T": 8191, "Hq": 16, "Hkv": 16, "D": 64, "style": "interleaved",
         "pad": 33, "maxpos": 8192},
        # The cache turn of a decode step: eight tokens written, and read back.
        {"name": "cache_decode_8", "kind": "cache", "B": 8, "Hkv": 8, "D": 128, "page": 16, "lo": 512, "hi": 4096,
         "nlo": 1, "nhi": 1, "read": "new", "lens": 1},
        # Sixteen whole prompts written and read back for the prefill attention.
        {"name": "cache_prompts_16", "kind": "cache", "B": 16, "Hkv": 8, "D": 128, "page": 16, "lo": 0, "hi": 0,
         "nlo": 256, "nhi": 8192, "read": "all", "lens": 2},
        # Chunked prefill: 512 more tokens for each of eight requests, all their keys read back, heads of 64.
        {"name": "cache_chunk_d64", "kind": "cache", "B": 8, "Hkv": 16, "D": 64, "page": 48, "lo": 512, "hi": 4096,
         "nlo": 511, "nhi": 513, "read": "all", "lens": 3},
        # Decode of eight requests at the repository's GQA lengths.
        {"name": "decode_gqa", "kind": "decode", "B": 8, "Hq": 32, "Hkv": 8, "Lq": 1, "D": 128, "page": 16, "lo": 512,
         "hi": 4096, "lens": 1},
        # Decode at long contexts, 32k to 128k keys (the repository's long decode).
        {"name": "decode_long", "kind": "decode", "B": 4, "Hq": 32, "Hkv": 8, "Lq": 1, "D": 128, "page": 64,
         "lo": 32768, "hi": 131072, "lens": 4},
        # Many short requests of a model without grouped heads, D = 64, empty and one-key rows among them.
        {"name": "decode_short_d64", "kind": "decode", "B": 64, "Hq": 16, "Hkv": 16, "Lq": 1, "D": 64, "page": 32,
         "lo": 0, "hi": 700, "lens": 5},
        # Eight draft tokens for each of eight requests, checked at once.
        {"name": "decode_multi_gqa", "kind": "decode", "B": 8, "Hq": 32, "Hkv": 8, "Lq": 8, "D": 128, "page": 16,
         "lo": 512, "hi": 4096, "lens": 6},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["pages", "norm", "cache", "decode", "decode"])
    lens = rng.randrange(1 << 20)
    D = rng.choice([64, 128, 128])
    Hkv, group = rng.choice([(1, 8), (2, 4), (4, 7), (4, 4), (8, 1), (8, 2), (8, 4), (16, 1), (5, 3), (4, 8)])
    if kind == "pages":
        B = _log(rng, 1, 256)
        hi = _log(rng, 1, 8192)
        nhi = rng.choice([1, rng.randint(2, 8), _log(rng, 16, 4096)])
        nhi = max(1, min(nhi, 131072 // B))
        return {"kind": kind, "B": B, "page": rng.choice([16, 32, 48, 64, 256]), "lo": 0, "hi": hi,
                "nlo": rng.randint(0, nhi), "nhi": nhi, "lens": lens}
    if kind == "norm":
        T = _log(rng, 1, 32768)
        return {"kind": kind, "T": T, "Hq": Hkv * group, "Hkv": Hkv, "D": D,
                "style": rng.choice(["half", "interleaved"]), "pad": rng.choice([0, 0, rng.randint(1, 64)]),
                "maxpos": _log(rng, 64, 131072)}
    if kind == "cache":
        B = _log(rng, 1, 64)
        nhi = rng.choice([1, _log(rng, 2, 4096)])
        nhi = max(1, min(nhi, 65536 // B))
        hi = max(1, min(_log(rng, 16, 8192), 131072 // B))
        return {"kind": kind, "B": B, "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 48, 64, 256]), "lo": 0,
                "hi": hi, "nlo": rng.randint(0, nhi), "nhi": nhi, "read": rng.choice(["new", "all"]), "lens": lens}
    B = _log(rng, 1, 64)
    hi = max(1, min(_log(rng, 8, 131072), 262144 // B))
    Lq = rng.choice([1, 1, 1, rng.randint(2, 8)])
    return {"kind": kind, "B": B, "Hq": Hkv * group, "Hkv": Hkv, "Lq": Lq, "D": D,
            "page": rng.choice([16, 32, 48, 64, 256]), "lo": rng.choice([0, hi // 2]), "hi": hi, "lens": lens}


# ---------------------------------------------------------------- lengths of a case (the same for every seed)

def _lens(c):
    """Cached keys of every request, and the tokens that come to them."""
    r = random.Random(c["lens"])
    a = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    n = [r.randint(c["nlo"], c["nhi"]) for _ in range(c["B"])] if "nlo" in c else [0] * c["B"]
    if c["kind"] == "decode":
        if c["lo"] == 0 and c["B"] > 2:
            a[0], a[1] = 0, 1  # a request without keys, one with a single key
        a[-1] = c["hi"]
    elif sum(n) == 0:
        n[0] = 1
    return a, n


def _pages(n, page):
    return -(-n // page)


def work(c):
    if c["kind"] == "norm":
        el = (c["T"] - c["pad"]) * (c["Hq"] + c["Hkv"]) * c["D"] if c["T"] > c["pad"] else c["D"]
        pos = min(c["maxpos"], c["T"])
        return {"bytes": 4 * el + pos * c["D"] * 4 + 4 * c["T"], "flops": 9 * el}
    a, n = _lens(c)
    if c["kind"] == "pages":
        moved = sum(_pages(x + y, c["page"]) - _pages(x, c["page"]) for x, y in zip(a, n))
        # grow: lengths in and out, slots and positions, the new entries and their pages; shrink: the way back
        return {"bytes": 2 * 12 * c["B"] + 8 * sum(n) + 4 * (c["B"] + 1) + 2 * 8 * moved, "flops": 0}
    D, H = c["D"], c["Hkv"]
    row = D + D // 8  # bytes of one key's K and V codes and parameters, of one head
    if c["kind"] == "cache":
        new, read = sum(n), sum(n) if c["read"] == "new" else sum(a) + sum(n)
        return {"bytes": H * (new * (4 * D + row) + read * (4 * D + row)) + 4 * new, "flops": 2 * D * H * (6 * new + 2 * read)}
    keys = sum(a)
    return {"bytes": keys * H * row + 4 * c["B"] * c["Hq"] * c["Lq"] * (D + 1), "flops": 4 * keys * c["Hq"] * c["Lq"] * D}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _table(a, page, num_pages, width, g):
    """Block table of requests that hold a[b] keys, -1 past their pages, and the pages nobody holds."""
    perm = torch.randperm(num_pages, generator=g, device=DEV, dtype=torch.int32)
    used = _ints([_pages(x, page) for x in a])
    at = torch.arange(width, device=DEV)[None, :]
    first = torch.cumsum(used, 0)[:, None] - used[:, None]
    idx = torch.where(at < used[:, None], first + at, 0)
    table = torch.where(at < used[:, None], perm[idx], -1).to(torch.int32).contiguous()
    total = sum(_pages(x, page) for x in a)
    free = torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)
    free[:num_pages - total] = perm[total:]
    return table, free, _ints([num_pages - total])


def _pool(num_pages, Hkv, page, D, g):
    """A pool whose codes and parameters are those of normally distributed rows (K with a few strong channels)."""
    G, tiles = D // 64, num_pages * Hkv * (page // 16)
    tile = 16 * (D + 8 * G)
    pool = torch.empty(tiles, tile, dtype=torch.uint8, device=DEV)
    step = 1 << 15
    for t0 in range(0, tiles, step):
        n = min(step, tiles - t0)
        codes = torch.randn(n, 16 * 2 * D, generator=g, device=DEV).mul_(3.0).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        pool[t0:t0 + n, :16 * D] = codes[:, 0::2] | (codes[:, 1::2] << 4)
        s = torch.rand(n, 2, 16, G, generator=g, device=DEV) * 0.25 + 0.2
        m = -s * (7.5 + torch.randn(n, 2, 16, G, generator=g, device=DEV))
        pool[t0:t0 + n, 16 * D:] = torch.stack([s, m], -1).half().view(n, -1).view(torch.uint8)
    return pool.view(num_pages, Hkv, page // 16, tile)


def _tables(maxpos, D):
    inv = 10000.0 ** (-torch.arange(0, D // 2, dtype=torch.float64, device=DEV) * 2.0 / D)
    ang = torch.arange(maxpos, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cos(ang).float(), torch.sin(ang).float()


def prepare(c, seed):
    g = _gen(seed)
    if c["kind"] == "norm":
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV)
        qkv *= torch.exp(torch.randn(T, 1, 1, generator=g, device=DEV))
        qkv = qkv.to(torch.bfloat16)
        w = (1 + 0.2 * torch.randn(2, D, generator=g, device=DEV)).to(torch.bfloat16)
        start = int(torch.randint(0, c["maxpos"], (1,), generator=g, device=DEV))
        pos = (torch.arange(T, device=DEV) + start) % c["maxpos"]
        if T > c["pad"]:
            pos[T - c["pad"]:] = -1  # rows of a batch padded to a captured size
        cos, sin = _tables(c["maxpos"], D)
        out = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV), torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device=DEV)
        return {"c": c, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "wq": w[0], "wk": w[1], "pos": pos.to(torch.int32),
                "cos": cos, "sin": sin, "q_out": out[0], "k_out": out[1]}
    a, n = _lens(c)
    page = c["page"]
    after = [x + y for x, y in zip(a, n)]
    width = max(1, max(_pages(x, page) for x in after))
    num_pages = sum(_pages(x, page) for x in after) + 3
    if c["kind"] == "pages":
        table, free, count = _table(a, page, num_pages, width, g)
        T = sum(n)
        return {"c": c, "lens": _ints(a), "old": _ints(a), "new": _ints(n), "table": table, "free": free, "count": count,
                "slots": torch.empty(T, dtype=torch.int32, device=DEV), "pos": torch.empty(T, dtype=torch.int32, device=DEV),
                "cu": torch.empty(c["B"] + 1, dtype=torch.int32, device=DEV)}
    D, Hkv = c["D"], c["Hkv"]
    table, _, _ = _table(after, page, num_pages, width, g)
    pool = _pool(num_pages, Hkv, page, D, g)
    if c["kind"] == "decode":
        q = torch.randn(c["B"], c["Hq"], c["Lq"], D, generator=g, device=DEV).to(torch.bfloat16)
        q = q if c["Lq"] > 1 else q[:, :, 0].contiguous()
        return {"c": c, "q": q, "pool": pool, "table": table, "lens": _ints(a), "out": torch.empty_like(q),
                "lse": torch.empty(q.shape[:-1], dtype=torch.float32, device=DEV)}
    T = sum(n)
    kv = torch.randn(T, 2 * Hkv, D, generator=g, device=DEV)
    kv *= torch.exp(0.5 * torch.randn(1, 2 * Hkv, D, generator=g, device=DEV))  # channels of unlike sizes
    kv = kv.to(torch.bfloat16)
    row = torch.repeat_interleave(torch.arange(c["B"], device=DEV), _ints(n).long(), output_size=T)
    first = torch.cumsum(_ints(n), 0) - _ints(n)
    pos = _ints(a)[row] + torch.arange(T, device=DEV) - first[row]
    slots = table[row, pos // page] * page + pos % page
    read = n if c["read"] == "new" else after
    cu = torch.zeros(c["B"] + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(_ints(read), 0)
    return {"c": c, "k": kv[:, :Hkv], "v": kv[:, Hkv:], "slots": slots.to(torch.int32), "pool": pool, "table": table,
            "cu": cu, "starts": _ints(a) if c["read"] == "new" else None, "total": sum(read),
            "k_out": torch.empty(sum(read), Hkv, D, dtype=torch.bfloat16, device=DEV),
            "v_out": torch.empty(sum(read), Hkv, D, dtype=torch.bfloat16, device=DEV)}


# ---------------------------------------------------------------- plain forms

def _page_step(s, page, keep, new):
    """Give back the pages past the kept and new keys, take pages for the rest, list the new tokens' slots."""
    lens, table, free, count = s["lens"], s["table"], s["free"], s["count"]
    a = lens.long()
    c = a if keep is None else keep.long()
    n = torch.zeros_like(a) if new is None else new.long()
    have, need = (a + page - 1) // page, (c + n + page - 1) // page
    at = torch.arange(table.shape[1], device=DEV)[None, :]
    gone = (at >= need[:, None]) & (at < have[:, None])
    taken = (at >= have[:, None]) & (at < need[:, None])
    given = table.flatten().flip(0)[gone.flatten().flip(0)]
    top = count.long()
    free[top + torch.arange(given.numel(), device=DEV)] = given
    table[gone] = -1
    top = top + given.numel()
    k = torch.cumsum(taken.flatten(), 0).view_as(taken) - 1
    table.copy_(torch.where(taken, free[(top - 1 - k).clamp(0, free.numel() - 1)], table))
    count.copy_(top - taken.sum())
    lens.copy_(c + n)
    cu = torch.zeros(a.numel() + 1, dtype=torch.int64, device=DEV)
    cu[1:] = torch.cumsum(n, 0)
    if new is None:
        return None, None, cu.to(torch.int32)
    i = torch.arange(s["slots"].numel(), device=DEV)
    row = torch.searchsorted(cu[1:], i, right=True)
    inside = i < cu[-1]
    row = row.clamp(max=a.numel() - 1)
    pos = c[row] + i - cu[row]
    slot = table[row, (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page
    return torch.where(inside, slot, -1).to(torch.int32), torch.where(inside, pos, -1).to(torch.int32), cu.to(torch.int32)


def _norm_rope(x, w, out, s):
    c = s["c"]
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
    pos = s["pos"].long()
    cos, sin = s["cos"][pos.clamp(min=0)][:, None], s["sin"][pos.clamp(min=0)][:, None]
    if c["style"] == "half":
        a, b = y[..., :c["D"] // 2], y[..., c["D"] // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.where((pos >= 0)[:, None, None], y.to(torch.bfloat16), out)


def _parts(pool, D):
    """Views of the pool's K codes, V codes [page, head, tile, group, key, byte], and parameters [.., key, group, 2]."""
    G, half = D // 64, 8 * D
    codes = pool[..., :half].unflatten(-1, (G, 16, 32)), pool[..., half:2 * half].unflatten(-1, (G, 16, 32))
    par = pool.view(torch.float16)
    mid = half + 16 * G * 2
    return codes, (par[..., half:mid].unflatten(-1, (16, G, 2)), par[..., mid:mid + 16 * G * 2].unflatten(-1, (16, G, 2)))


def _append(x, codes, par, slots, page):
    G = x.shape[-1] // 64
    y = torch.nan_to_num(x.float(), nan=0.0, posinf=F16_MAX, neginf=-F16_MAX).clamp(-F16_MAX, F16_MAX).unflatten(-1, (G, 64))
    lo, hi = y.amin(-1), y.amax(-1)
    m, s = lo.half(), ((hi - lo) / 15).half()
    at = (y.double() - m.double()[..., None]) / torch.where(s == 0, 1.0, s.double())[..., None]  # values next to a border
    u = torch.where((s == 0)[..., None], 0, torch.round(at).clamp(0, 15)).to(torch.uint8)
    slots = slots.long()
    pg, tile, row = slots // page, slots % page // 16, slots % 16
    codes[pg, :, tile, :, row] = u[..., 0::2] | (u[..., 1::2] << 4)
    par[pg, :, tile, row] = torch.stack([s, m], -1)


def _values(codes, par, pg, tile, row):
    """The rows (page, tile, key) of every head, in 32 bits: [rows, Hkv, D]."""
    b = codes[pg, :, tile, :, row]
    u = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
    p = par[pg, :, tile, row].float()
    return (u * p[..., 0:1] + p[..., 1:2]).flatten(-2)


def _cache(s):
    c, page = s["c"], s["c"]["page"]
    codes, par = _parts(s["pool"], c["D"])
    _append(s["k"], codes[0], par[0], s["slots"], page)
    _append(s["v"], codes[1], par[1], s["slots"], page)
    i = torch.arange(s["total"], device=DEV)
    cu = s["cu"].long()
    row = torch.searchsorted(cu[1:], i, right=True)
    pos = i - cu[row] + (0 if s["starts"] is None else s["starts"].long()[row])
    pg = s["table"].long()[row, pos // page]
    at = pg, pos % page // 16, pos % 16
    return {"k": _values(codes[0], par[0], *at).to(torch.bfloat16), "v": _values(codes[1], par[1], *at).to(torch.bfloat16)}


def _decode(s):
    c, page = s["c"], s["c"]["page"]
    B, Hkv, D, Lq, L = c["B"], c["Hkv"], c["D"], c["Lq"], max(1, c["hi"])
    group = c["Hq"] // Hkv
    codes, par = _parts(s["pool"], D)
    j = torch.arange(L, device=DEV)
    lens = s["lens"].long()
    pg = s["table"].long()[:, j // page].clamp(min=0).flatten()
    at = pg, (j % page // 16).repeat(B), (j % 16).repeat(B)
    k = _values(codes[0], par[0], *at).view(B, L, Hkv, D)
    x = torch.einsum("bhrd,blhd->bhrl", s["q"].float().view(B, Hkv, group * Lq, D), k) * D ** -0.5
    del k
    last = (lens[:, None] - Lq + torch.arange(Lq, device=DEV)).repeat(1, group)[:, None, :, None]
    x = torch.where(j <= last, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    del x
    l = p.sum(-1, keepdim=True)
    v = _values(codes[1], par[1], *at).view(B, L, Hkv, D)
    v = torch.where((j < lens[:, None])[..., None, None], v, 0.0)
    o = torch.einsum("bhrl,blhd->bhrd", p, v) / torch.where(l == 0, 1.0, l)
    return {"out": o.to(torch.bfloat16).view(s["q"].shape), "lse": (m + torch.log(l)).view(s["lse"].shape)}


def run(s):
    c = s["c"]
    if c["kind"] == "pages":
        # Tokens come to every request, then they are taken back (drafts refused, or the request released).
        if own:
            from attention_attn_fwd_06_gb300 import binding as attn

            attn.attn_page_step(s["lens"], s["table"], s["free"], s["count"], c["page"], new_lens=s["new"],
                                slots=s["slots"], positions=s["pos"], cu_new=s["cu"])
            attn.attn_page_step(s["lens"], s["table"], s["free"], s["count"], c["page"], keep_lens=s["old"])
            slots, pos, cu = s["slots"], s["pos"], s["cu"]
        else:
            slots, pos, cu = _page_step(s, c["page"], None, s["new"])
            _page_step(s, c["page"], s["old"], None)
        return {"slots": slots, "pos": pos, "cu": cu, "lens": s["lens"], "table": s["table"], "free": s["free"],
                "count": s["count"]}
    if c["kind"] == "norm":
        if own:
            from attention_attn_fwd_06_gb300 import binding as attn

            q, k = attn.attn_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], (s["cos"], s["sin"], c["style"]), s["pos"],
                                          eps=1e-6, q_out=s["q_out"], k_out=s["k_out"])
            return {"q": q, "k": k}
        return {"q": _norm_rope(s["q"], s["wq"], s["q_out"], s), "k": _norm_rope(s["k"], s["wk"], s["k_out"], s)}
    if c["kind"] == "cache":
        if own:
            from attention_attn_fwd_06_gb300 import binding as attn

            attn.attn_kv_append_q4(s["k"], s["v"], s["pool"], s["slots"])
            k, v = attn.attn_kv_gather_q4(s["pool"], s["table"], s["cu"], s["total"], kv_starts=s["starts"],
                                          k_out=s["k_out"], v_out=s["v_out"])
            return {"k": k, "v": v}
        return _cache(s)
    if own:
        from attention_attn_fwd_06_gb300 import binding as attn

        out, lse = attn.attn_decode_q4(s["q"], s["pool"], s["table"], s["lens"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    return _decode(s)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_row(pool, table, b, first, last, page, D, which):
    """Keys first..last-1 of request b, read tile by tile from the pool's bytes: [keys, Hkv, D] in 64 bits."""
    G = D // 64
    pages = table[b, first // page:_pages(last, page)].long()
    tiles = pool[pages].transpose(1, 2).flatten(0, 1)  # [tiles, Hkv, bytes]
    codes = tiles[..., which * 8 * D:(which + 1) * 8 * D].reshape(*tiles.shape[:2], G, 16, 32)
    base = 16 * D + which * 64 * G
    par = tiles[..., base:base + 64 * G].contiguous().view(torch.float16).double().view(*tiles.shape[:2], 16, G, 2)
    x = torch.empty(tiles.shape[0], 16, tiles.shape[1], G, 64, dtype=torch.float64, device=DEV)
    x[..., 0::2] = (codes & 15).double().permute(0, 3, 1, 2, 4)
    x[..., 1::2] = (codes >> 4).double().permute(0, 3, 1, 2, 4)
    par = par.permute(0, 2, 1, 3, 4)
    x.mul_(par[..., 0:1]).add_(par[..., 1:2])
    skip = first - first // page * page
    return x.view(-1, tiles.shape[1], D)[skip:skip + last - first]


def exact(c, seed):
    if c["kind"] == "pages":
        return None
    s = prepare(c, seed)
    if c["kind"] == "norm":
        pos, got = s["pos"].long(), {}
        for name, x, w in (("q", s["q"], s["wq"]), ("k", s["k"], s["wk"])):
            y = x.double()
            y = y / torch.sqrt((y ** 2).sum(-1, keepdim=True) / c["D"] + 1e-6) * w.double()
            pair = torch.complex(*(y.chunk(2, -1) if c["style"] == "half" else (y[..., ::2], y[..., 1::2])))
            turn = torch.complex(s["cos"].double(), s["sin"].double())[pos.clamp(min=0)][:, None]
            pair = pair * turn * (pos >= 0)[:, None, None]
            got[name] = torch.cat([pair.real, pair.imag], -1) if c["style"] == "half" else torch.view_as_real(pair).flatten(-2)
        return got
    a, n = _lens(c)
    page, D, Hkv = c["page"], c["D"], c["Hkv"]
    if c["kind"] == "cache":
        parts = {"k": [], "v": []}
        for which, name in enumerate("kv"):
            x = s[name].double().nan_to_num(nan=0.0).clamp(-F16_MAX, F16_MAX).view(-1, Hkv, D // 64, 64)
            m = x.min(-1, keepdim=True).values.float().half().double()
            sc = ((x.max(-1, keepdim=True).values - x.min(-1, keepdim=True).values) / 15).float().half().double()
            u = torch.where(sc > 0, torch.round((x - m) / torch.where(sc > 0, sc, 1.0)), 0.0).clamp(0, 15)
            new, done = (u * sc + m).view(-1, Hkv, D), 0
            for b in range(c["B"]):
                if c["read"] == "all" and a[b]:
                    parts[name].append(_exact_row(s["pool"], s["table"], b, 0, a[b], page, D, which))
                parts[name].append(new[done:done + n[b]])
                done += n[b]
        return {name: torch.cat(v) for name, v in parts.items()}
    group, Lq = c["Hq"] // Hkv, c["Lq"]
    q = s["q"].double().view(c["B"], Hkv, group, Lq, D)
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        if not a[b]:
            continue
        k = _exact_row(s["pool"], s["table"], b, 0, a[b], page, D, 0)
        x = torch.einsum("hgtd,lhd->hgtl", q[b], k) / math.sqrt(D)
        for t in range(Lq):
            see = a[b] - Lq + t + 1
            if see > 0:
                lse[b, :, :, t] = torch.logsumexp(x[:, :, t, :see], -1)
                x[:, :, t, :see] = torch.exp(x[:, :, t, :see] - lse[b, :, :, t, None])
            x[:, :, t, max(see, 0):] = 0.0
        del k
        out[b] = torch.einsum("hgtl,lhd->hgtd", x, _exact_row(s["pool"], s["table"], b, 0, a[b], page, D, 1))
    return {"out": out.view(s["q"].shape), "lse": lse.view(s["lse"].shape)}
