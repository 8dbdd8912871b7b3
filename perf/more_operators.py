"""Cases of a draft step over a paged bf16 KV cache: rotary tables, keys and values into the pages with the rotation on the
way, attention of every sequence's drafted tokens over the pages, and the decision which drafts stand.  Every case has a
plain torch form beside the framework's call.

A page pool is [num_pages, Hkv, page_size, D] for keys and another for values; slot = page * page_size + offset.  The step's
tokens are packed, sequence after sequence: cu[b] .. cu[b + 1] - 1 are those of sequence b.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # 4096 rows of tables, made when a model is loaded or its requests grow longer: every dim of a head of 128.
        {"name": "tables_4k", "kind": "tables", "rows": 4096, "R": 128, "base": 10000.0, "scaling": "none", "factor": 1.0,
         "context": 4096, "low": 1.0, "high": 4.0, "amplitude": 1.0, "reach": 8192},
        # A model of 8k positions stretched to 128k, slow pairs interpolated.
        {"name": "tables_128k_turns", "kind": "tables", "rows": 131072, "R": 128, "base": 500000.0, "scaling": "turns",
         "factor": 8.0, "context": 8192, "low": 1.0, "high": 4.0, "amplitude": 1.0, "reach": 1 << 18},
        # Tables that grow with the longest request: another 8191 rows far out, three quarters of a head of 64.
        {"name": "tables_far_d48", "kind": "tables", "rows": 8191, "R": 48, "base": 10000.0, "scaling": "index",
         "factor": 32.0, "context": 4096, "low": 1.0, "high": 32.0, "amplitude": 1.3466, "reach": 1 << 20},
        # One token of each of eight requests out of a fused projection: latency.
        {"name": "append_decode_8", "kind": "append", "T": 8, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "page": 16,
         "style": "half", "pad": 0, "maxpos": 4096, "q": True, "lens": 1},
        # The prompts of a ragged prefill batch, for which the packed keys are wanted too: bandwidth.
        {"name": "append_prompts_64k", "kind": "append", "T": 65536, "Hq": 32, "Hkv": 8, "D": 128, "R": 128, "page": 16,
         "style": "half", "pad": 0, "maxpos": 8192, "q": True, "lens": 2},
        # Half of each head turned, interleaved pairs, a batch padded for a graph.
        {"name": "append_d64_partial", "kind": "append", "T": 8191, "Hq": 16, "Hkv": 16, "D": 64, "R": 32, "page": 48,
         "style": "interleaved", "pad": 33, "maxpos": 8192, "q": True, "lens": 3},
        # Eight drafted tokens of each of eight requests at the repository's GQA lengths.
        {"name": "draft_gqa_8", "kind": "decode", "B": 8, "Hq": 32, "Hkv": 8, "nlo": 8, "nhi": 8, "D": 128, "page": 16,
         "lo": 512, "hi": 4096, "lens": 4},
        # The same at long contexts, 32k to 128k keys.
        {"name": "draft_long", "kind": "decode", "B": 4, "Hq": 32, "Hkv": 8, "nlo": 8, "nhi": 8, "D": 128, "page": 64,
         "lo": 32768, "hi": 131072, "lens": 5},
        # Many short requests, one to five tokens each, no grouped heads, D = 64; empty and one-key requests among them.
        {"name": "draft_short_d64", "kind": "decode", "B": 64, "Hq": 16, "Hkv": 16, "nlo": 1, "nhi": 5, "D": 64, "page": 48,
         "lo": 0, "hi": 700, "lens": 6},
        # Four drafts of each of eight requests.
        {"name": "verify_8", "kind": "verify", "B": 8, "K": 4, "V": 32000, "dtype": "fp32", "packed": False, "point": False,
         "ragged": False, "lens": 7},
        # Up to eight drafts of 64 requests over a large vocabulary, packed as the step's tokens are.
        {"name": "verify_64_packed", "kind": "verify", "B": 64, "K": 8, "V": 131072, "dtype": "fp32", "packed": True,
         "point": False, "ragged": True, "lens": 8},
        # Drafts looked up in the prompt (no distribution of their own), an odd vocabulary, probabilities in 16 bits.
        {"name": "verify_lookup_37", "kind": "verify", "B": 37, "K": 6, "V": 50001, "dtype": "bf16", "packed": False,
         "point": True, "ragged": True, "lens": 9},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["tables", "append", "decode", "decode", "verify", "verify"])
    lens = rng.randrange(1 << 20)
    D = rng.choice([64, 128, 128])
    Hkv, group = rng.choice([(1, 8), (2, 4), (4, 7), (4, 4), (8, 1), (8, 2), (8, 4), (16, 1), (5, 3), (4, 8)])
    if kind == "tables":
        R = 16 * rng.randint(1, 8)
        reach = _log(rng, 4096, 1 << 20)
        return {"kind": kind, "rows": min(_log(rng, 1, 65536), reach // 2), "R": R, "base": rng.choice([10000.0, 500000.0, 1e6]),
                "scaling": rng.choice(["none", "linear", "base", "turns", "index"]), "factor": rng.choice([1.5, 2.0, 8.0, 40.0]),
                "context": rng.choice([2048, 4096, 8192]), "low": 1.0, "high": rng.choice([4.0, 32.0]),
                "amplitude": rng.choice([1.0, 1.2]), "reach": reach}
    if kind == "append":
        T = _log(rng, 1, 32768)
        return {"kind": kind, "T": T, "Hq": Hkv * group, "Hkv": Hkv, "D": D,
                "R": rng.choice([D, D, 16 * rng.randint(1, D // 16)]), "page": rng.choice([8, 16, 32, 48, 64, 256]),
                "style": rng.choice(["half", "interleaved", "none"]), "pad": rng.choice([0, 0, rng.randint(1, 64)]),
                "maxpos": _log(rng, 64, 131072), "q": rng.choice([True, True, False]), "lens": lens}
    if kind == "decode":
        B = _log(rng, 1, 64)
        hi = max(1, min(_log(rng, 8, 131072), 262144 // B))
        nhi = rng.randint(1, min(16, 128 // group))
        return {"kind": kind, "B": B, "Hq": Hkv * group, "Hkv": Hkv, "nlo": rng.choice([0, 1, nhi]), "nhi": nhi, "D": D,
                "page": rng.choice([8, 16, 32, 48, 64, 256]), "lo": rng.choice([0, hi // 2]), "hi": hi, "lens": lens}
    B, K = _log(rng, 1, 128), rng.randint(1, 12)
    V = max(7, min(_log(rng, 100, 262144), (60 << 20) // (B * (2 * K + 1))))
    return {"kind": kind, "B": B, "K": K, "V": V, "dtype": rng.choice(["fp32", "fp32", "bf16"]),
            "packed": rng.choice([False, True]), "point": rng.choice([False, False, True]),
            "ragged": rng.choice([False, True]), "lens": lens}


# ---------------------------------------------------------------- lengths of a case (the same for every seed)

def _lens(c):
    """decode: every request's keys (the new tokens' own among them) and new tokens; verify: its drafts."""
    r = random.Random(c["lens"])
    if c["kind"] == "verify":
        n = [r.randint(0, c["K"]) if c["ragged"] else c["K"] for _ in range(c["B"])]
        n[-1] = c["K"]
        return None, n
    a = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    n = [r.randint(c["nlo"], c["nhi"]) for _ in range(c["B"])]
    if c["lo"] == 0 and c["B"] > 2:
        a[0], a[1] = 0, 1  # a request without keys, one with a single key
    a[-1], n[-1] = c["hi"], c["nhi"]
    return a, n


def _pages(n, page):
    return -(-n // page)


def _draft_rows(c):
    """Rows of the target's probabilities and of the drafts' own."""
    n = _lens(c)[1]
    return (sum(n) + c["B"] if c["packed"] else c["B"] * (c["K"] + 1)), c["B"] * c["K"]


def work(c):
    if c["kind"] == "tables":
        return {"bytes": 4 * c["rows"] * c["R"], "flops": 4 * c["rows"] * c["R"]}
    if c["kind"] == "append":
        T = max(1, c["T"] - c["pad"])
        heads = c["Hq"] * c["q"] + c["Hkv"]
        return {"bytes": 4 * T * (heads + c["Hkv"]) * c["D"] + 4 * min(c["maxpos"], T) * c["R"] * (c["style"] != "none") + 8 * c["T"],
                "flops": 3 * T * heads * c["R"]}
    a, n = _lens(c)
    if c["kind"] == "decode":
        keys = sum(x for x, y in zip(a, n) if y)
        el = sum(n) * c["Hq"]
        return {"bytes": keys * c["Hkv"] * c["D"] * 4 + 4 * el * (c["D"] + 1),
                "flops": 4 * c["Hq"] * c["D"] * sum(x * y for x, y in zip(a, n))}
    size = 4 if c["dtype"] == "fp32" else 2
    rows = c["B"] * (1 if c["point"] else 2)  # (where every draft stands the draft's row is not read: few of them)
    return {"bytes": rows * c["V"] * size + sum(n) * (4 + 4 + 2 * size), "flops": 3 * rows * c["V"]}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(n):
    return torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), torch.cumsum(_ints(n), 0).to(torch.int32)])


def prepare(c, seed):
    g = _gen(seed)
    if c["kind"] == "tables":
        start = random.Random(seed).randint(0, c["reach"] - c["rows"])
        shape = c["rows"], c["R"] // 2
        return {"c": c, "start": start, "cos": torch.empty(shape, device=DEV), "sin": torch.empty(shape, device=DEV)}
    if c["kind"] == "append":
        T, Hq, Hkv, D, page = c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV)
        qkv *= torch.exp(0.5 * torch.randn(1, Hq + 2 * Hkv, D, generator=g, device=DEV))  # channels of unlike sizes
        qkv = qkv.to(torch.bfloat16)
        # runs of consecutive positions on pages in no order; padding at the end
        num_pages = _pages(T, page) + 3
        perm = torch.randperm(num_pages, generator=g, device=DEV)
        i = torch.arange(T, device=DEV)
        slots = perm[i // page] * page + i % page
        start = int(torch.randint(0, c["maxpos"], (1,), generator=g, device=DEV))
        pos = (i + start) % c["maxpos"]
        if T > c["pad"] > 0:
            slots[T - c["pad"]:] = -1
            pos[T - c["pad"]:] = -1
        inv = 10000.0 ** (-torch.arange(0, c["R"] // 2, dtype=torch.float64, device=DEV) * 2.0 / c["R"])
        ang = torch.arange(c["maxpos"], dtype=torch.float64, device=DEV)[:, None] * inv
        pools = [torch.empty(num_pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(2)]
        return {"c": c, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hkv], "v": qkv[:, Hq + Hkv:], "kpages": pools[0], "vpages": pools[1],
                "slots": slots.to(torch.int32), "pos": pos.to(torch.int32), "cos": torch.cos(ang).float(),
                "sin": torch.sin(ang).float(), "q_out": torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV)}
    a, n = _lens(c)
    if c["kind"] == "decode":
        D, Hkv, page = c["D"], c["Hkv"], c["page"]
        used = [_pages(x, page) for x in a]
        num_pages, width = sum(used) + 3, max(1, max(used))
        perm = torch.randperm(num_pages, generator=g, device=DEV, dtype=torch.int32)
        at, u = torch.arange(width, device=DEV)[None, :], _ints(used)[:, None]
        idx = torch.cumsum(_ints(used), 0)[:, None] - u + at
        table = torch.where(at < u, perm[idx.clamp(max=num_pages - 1)], -1).to(torch.int32).contiguous()
        pools = [torch.empty(num_pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV).normal_(generator=g) for _ in range(2)]
        T = sum(n)
        q = torch.empty(T, c["Hq"], D, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
        return {"c": c, "q": q, "kpages": pools[0], "vpages": pools[1], "table": table, "lens": _ints(a), "cu": _cu(n),
                "out": torch.zeros_like(q), "lse": torch.zeros(T, c["Hq"], dtype=torch.float32, device=DEV)}
    B, K, V = c["B"], c["K"], c["V"]
    dtype = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
    rows, _ = _draft_rows(c)
    n = _ints(n)
    logits = torch.randn(B * K, V, generator=g, device=DEV).mul_(3.0)
    q = torch.softmax(logits, -1)
    drafts = torch.multinomial(q, 1, generator=g).to(torch.int32).view(B, K)
    # the target's: near the draft's row of the same place
    if c["packed"]:
        row = torch.repeat_interleave(torch.arange(B, device=DEV), n.long() + 1, output_size=rows)
        place = torch.arange(rows, device=DEV) - (_cu(_lens(c)[1]).long()[:-1] + torch.arange(B, device=DEV))[row]
    else:
        row, place = torch.arange(rows, device=DEV) // (K + 1), torch.arange(rows, device=DEV) % (K + 1)
    p = logits[row * K + place.clamp(max=K - 1)]
    p = torch.softmax(p.add_(torch.randn(p.shape, generator=g, device=DEV).mul_(0.5)), -1).to(dtype)
    if c["packed"]:
        cu = _cu([x + 1 for x in _lens(c)[1]])
    else:
        cu, p = None, p.view(B, K + 1, V)
    return {"c": c, "drafts": drafts, "p": p, "q": None if c["point"] else q.to(dtype).view(B, K, V), "cu": cu,
            "n": None if c["packed"] else n, "u": torch.rand(B, K + 1, generator=g, device=DEV),
            "lens": n + 1 + torch.randint(0, 4096, (B,), generator=g, device=DEV, dtype=torch.int32),
            "tokens": torch.empty(B, K + 1, dtype=torch.int32, device=DEV), "accepted": torch.empty(B, dtype=torch.int32, device=DEV),
            "keep": torch.empty(B, dtype=torch.int32, device=DEV)}


# ---------------------------------------------------------------- plain forms

def _frequencies(c):
    """Radians a position, of every pair, in 64 bits."""
    R, s = c["R"], c["factor"]
    i = torch.arange(R // 2, dtype=torch.float64, device=DEV)
    base = c["base"] * s ** (R / (R - 2)) if c["scaling"] == "base" else c["base"]
    f = base ** (-2.0 * i / R)
    if c["scaling"] == "linear":
        return f / s
    if c["scaling"] == "turns":  # by the turns that a pair makes over the context
        keep = ((c["context"] * f / (2 * math.pi) - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
    elif c["scaling"] == "index":  # straight between the pairs that make `high` and `low` turns
        first = max(0, math.floor(R / 2 * math.log(c["context"] / (2 * math.pi * c["high"])) / math.log(base)))
        last = min(R - 1, math.ceil(R / 2 * math.log(c["context"] / (2 * math.pi * c["low"])) / math.log(base)))
        keep = 1 - ((i - first) / max(last - first, 0.001)).clamp(0, 1)
    else:
        return f
    return f * (keep + (1 - keep) / s)


def _tables(s):
    c = s["c"]
    pos = s["start"] + torch.arange(c["rows"], dtype=torch.float64, device=DEV)
    ang = pos[:, None] * _frequencies(c)
    return {"cos": (torch.cos(ang) * c["amplitude"]).float(), "sin": (torch.sin(ang) * c["amplitude"]).float()}


def _rotate(x, s):
    c = s["c"]
    y = x.float()
    if c["style"] == "none":
        return x
    pos, R = s["pos"].long().clamp(min=0), c["R"]
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    y, rest = y[..., :R], y[..., R:]
    if c["style"] == "half":
        a, b = y[..., :R // 2], y[..., R // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, rest], -1).to(torch.bfloat16)


def _append(s):
    c, page, slots = s["c"], s["c"]["page"], s["slots"].long()
    live = c["T"] - c["pad"] if c["T"] > c["pad"] else c["T"]
    at = slots[:live] // page, slice(None), slots[:live] % page
    s["kpages"][at] = _rotate(s["k"], s)[:live]
    s["vpages"][at] = s["v"][:live]
    got = {"kpages": s["kpages"], "vpages": s["vpages"]}
    if c["q"] and c["style"] != "none":
        got["q"] = torch.where((s["pos"] >= 0)[:, None, None], _rotate(s["q"], s), s["q_out"])
    return got


def _decode(s):
    c, page = s["c"], s["c"]["page"]
    B, Hkv, D, N, L = c["B"], c["Hkv"], c["D"], c["nhi"], max(1, c["hi"])
    group = c["Hq"] // Hkv
    cu, lens = s["cu"].long(), s["lens"].long()
    n = cu[1:] - cu[:-1]
    t = torch.arange(N, device=DEV)
    real = t < n[:, None]
    q = s["q"].float()[(cu[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)].view(B, N, Hkv, group, D)
    j = torch.arange(L, device=DEV)
    pg = s["table"].long()[:, j // page].clamp(min=0)
    k = s["kpages"][pg, :, j % page].float()  # [B, L, Hkv, D]
    x = torch.einsum("bthgd,blhd->bthgl", q, k) * D ** -0.5
    del k
    last = torch.where(real, lens[:, None] - n[:, None] + t, -1)[:, :, None, None, None]
    x = torch.where(j <= last, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    del x
    l = p.sum(-1, keepdim=True)
    v = s["vpages"][pg, :, j % page].float()
    v = torch.where((j < lens[:, None])[..., None, None], v, 0.0)
    o = torch.einsum("bthgl,blhd->bthgd", p, v) / torch.where(l == 0, 1.0, l)
    at = real.flatten().nonzero()[:, 0]
    return {"out": o.to(torch.bfloat16).reshape(B * N, c["Hq"], D)[at], "lse": (m + torch.log(l)).reshape(B * N, c["Hq"])[at]}


def _verify(s):
    c, K, V = s["c"], s["c"]["K"], s["c"]["V"]
    b = torch.arange(c["B"], device=DEV)[:, None]
    i = torch.arange(K, device=DEV)[None, :]
    if c["packed"]:
        first, n = s["cu"].long()[:-1], (s["cu"][1:] - s["cu"][:-1]).long() - 1
    else:
        first, n = b[:, 0] * (K + 1), s["n"].long()
    p = s["p"].view(-1, V)
    x = s["drafts"].long()
    px = p[(first[:, None] + i).clamp(max=p.shape[0] - 1), x].double()
    qx = 1.0 if s["q"] is None else s["q"][b, i, x].double()
    stands = (s["u"][:, :K].double() * qx < px) & (i < n[:, None])
    accepted = torch.cumprod(stands.int(), 1).sum(1)
    refused = accepted < n
    w = p[first + accepted].double()
    at = accepted.clamp(max=K - 1)
    if s["q"] is None:
        less = torch.where(torch.arange(V, device=DEV) == x[b[:, 0], at][:, None], w, 0.0)
    else:
        less = s["q"][b[:, 0], at].double()
    rest = (w - torch.where(refused[:, None], less, 0.0)).clamp(min=0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w)
    total = torch.cumsum(rest, -1)
    token = (total <= s["u"][:, K:].double() * total[:, -1:]).sum(-1)
    place = torch.arange(K + 1, device=DEV)[None, :]
    tokens = torch.where(place < accepted[:, None], torch.cat([x, x[:, :1]], 1), -1)
    tokens = torch.where(place == accepted[:, None], token[:, None], tokens)
    return {"tokens": tokens.to(torch.int32), "accepted": accepted.to(torch.int32),
            "keep": (s["lens"] - (n - accepted)).to(torch.int32)}


def run(s):
    c = s["c"]
    if c["kind"] == "tables":
        if own:
            from attention_attn_fwd_06_gb300 import binding as attn

            scaling = {"none": None, "linear": ("linear", c["factor"]), "base": ("base", c["factor"])}.get(
                c["scaling"], (c["scaling"], c["factor"], c["context"], c["low"], c["high"]))
            cos, sin = attn.attn_rope_tables(c["rows"], c["R"], base=c["base"], scaling=scaling, amplitude=c["amplitude"],
                                             start=s["start"], cos=s["cos"], sin=s["sin"])
            return {"cos": cos, "sin": sin}
        return _tables(s)
    if c["kind"] == "append":
        if own:
            from attention_attn_fwd_06_gb300 import binding as attn

            turned = c["style"] != "none"
            q = {"q": s["q"], "q_out": s["q_out"]} if c["q"] and turned else {}
            attn.attn_kv_append_paged(s["k"], s["v"], s["kpages"], s["vpages"], s["slots"],
                                      rope=(s["cos"], s["sin"], c["style"]) if turned else None,
                                      positions=s["pos"] if turned else None, **q)
            return {"kpages": s["kpages"], "vpages": s["vpages"], **({"q": s["q_out"]} if q else {})}
        return _append(s)
    if c["kind"] == "decode":
        if own:
            from attention_attn_fwd_06_gb300 import binding as attn

            out, lse = attn.attn_decode_multi_paged(s["q"], s["kpages"], s["vpages"], s["table"], s["lens"], s["cu"], c["nhi"],
                                                    out=s["out"], lse=s["lse"])
            return {"out": out, "lse": lse}
        return _decode(s)
    if own:
        from attention_attn_fwd_06_gb300 import binding as attn

        tokens, accepted, keep = attn.attn_verify_drafts(
            s["drafts"], s["p"], s["u"], draft_probs=s["q"], cu_target=s["cu"], draft_lens=s["n"], kv_lens=s["lens"],
            tokens=s["tokens"], accepted=s["accepted"], keep_lens=s["keep"])
        return {"tokens": tokens, "accepted": accepted, "keep": keep}
    return _verify(s)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(c, seed):
    if c["kind"] == "verify":
        return None
    s = prepare(c, seed)
    if c["kind"] == "tables":
        R, half = c["R"], c["R"] // 2
        turns = []
        for i in range(half):  # turns a position
            base = c["base"]
            if c["scaling"] == "base":
                base *= math.exp(math.log(c["factor"]) * R / (R - 2.0))
            f = math.exp(-math.log(base) * i / half)
            part = 1.0  # how much of the pair keeps its speed
            if c["scaling"] == "linear":
                part = 0.0
            elif c["scaling"] == "turns":
                part = min(1.0, max(0.0, (c["context"] * f / math.tau - c["low"]) / (c["high"] - c["low"])))
            elif c["scaling"] == "index":
                lo, hi = (half * math.log(c["context"] / math.tau / x) / math.log(base) for x in (c["high"], c["low"]))
                lo, hi = max(0, math.floor(lo)), min(R - 1, math.ceil(hi))
                part = 1.0 - min(1.0, max(0.0, (i - lo) / max(0.001, hi - lo)))
            turns.append((f * part + f * (1.0 - part) / c["factor"]) / math.tau)
        pos = torch.arange(s["start"], s["start"] + c["rows"], dtype=torch.float64, device=DEV)
        t = torch.outer(pos, torch.tensor(turns, dtype=torch.float64, device=DEV))
        z = torch.polar(torch.full_like(t, c["amplitude"]), (t - torch.round(t)) * math.tau)
        return {"cos": z.real.contiguous(), "sin": z.imag.contiguous()}
    if c["kind"] == "append":
        page, R, T = c["page"], c["R"], c["T"]
        got = {"kpages": s["kpages"].double(), "vpages": s["vpages"].double()}
        live = (s["slots"] >= 0).nonzero()[:, 0]
        where = s["slots"].long()[live]
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long().clamp(min=0)][:, None]
        rows = {}
        for name in ("k", "v", "q"):
            y = s[name].double()
            if name != "v" and c["style"] != "none":
                head = y[..., :R]
                pair = torch.complex(*(z.contiguous() for z in (head.chunk(2, -1) if c["style"] == "half" else
                                                                (head[..., ::2], head[..., 1::2])))) * turn
                head = torch.cat([pair.real, pair.imag], -1) if c["style"] == "half" else torch.view_as_real(pair).flatten(-2)
                y = torch.cat([head, y[..., R:]], -1)
            rows[name] = y
        for name in ("k", "v"):
            flat = got[name + "pages"].transpose(1, 2).reshape(-1, c["Hkv"], c["D"])  # by slot
            flat[where] = rows[name][live]
            got[name + "pages"] = flat.view(-1, page, c["Hkv"], c["D"]).transpose(1, 2)
        if c["q"] and c["style"] != "none":
            got["q"] = rows["q"] * (s["pos"] >= 0)[:, None, None]
        return got
    a, n = _lens(c)
    page, D, Hkv, group = c["page"], c["D"], c["Hkv"], c["Hq"] // c["Hkv"]
    q = s["q"].double().view(-1, Hkv, group, D)
    out, lse = torch.zeros_like(q), torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=DEV)
    done = 0
    for b in range(c["B"]):
        mine = slice(done, done + n[b])
        done += n[b]
        if not a[b] or not n[b]:
            continue
        pages = s["table"][b, :_pages(a[b], page)].long()
        k, v = (s[name][pages].transpose(1, 2).reshape(-1, Hkv, D)[:a[b]].double() for name in ("kpages", "vpages"))
        x = torch.einsum("thgd,lhd->thgl", q[mine], k) / math.sqrt(D)
        for t in range(n[b]):
            x[t, :, :, max(0, a[b] - n[b] + t + 1):] = -math.inf
        lse[mine] = torch.logsumexp(x, -1)
        x = torch.exp(x - lse[mine].clamp(min=-1e300)[..., None])
        out[mine] = torch.einsum("thgl,lhd->thgd", x, v)
    return {"out": out.view(-1, c["Hq"], D), "lse": lse.view(-1, c["Hq"])}
