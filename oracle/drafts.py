"""Plain forms of a draft step over a paged bf16 cache -- TEST INFRASTRUCTURE ONLY.

``rope_frequencies`` / ``rope_table_rows`` are the rotary tables in fp64, ``rotate_part`` the rotation of a head's first
dims, ``append_paged`` writes rows into pages, ``decode_multi_paged`` is :func:`oracle.attention_head` over each sequence's
keys read page by page, ``verify_drafts`` decides drafts in exact integers.  Nothing here shares code with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

from .sdpa import attention_head, to_f64


def rope_frequencies(rotary_dim, base=10000.0, scaling=None):
    """Radians a position of each of the rotary_dim / 2 pairs."""
    R, out = rotary_dim, []
    kind = scaling[0] if scaling else None
    for i in range(R // 2):
        b = base
        if kind == "base":
            b = base * scaling[1] ** (R / (R - 2))
        f = math.exp(-2.0 * i / R * math.log(b))
        if kind == "linear":
            f = f / scaling[1]
        elif kind in ("turns", "index"):
            _, factor, context, low, high = scaling
            if kind == "turns":
                g = (context * f / (2 * math.pi) - low) / (high - low)
            else:
                def pair(turns):
                    return R / 2 * math.log(context / (2 * math.pi * turns)) / math.log(base)
                a, z = max(0, math.floor(pair(high))), min(R - 1, math.ceil(pair(low)))
                g = 1 - (i - a) / max(z - a, 0.001)
            g = min(1.0, max(0.0, g))
            f = f * g + f * (1 - g) / factor
        out.append(f)
    return np.array(out)


def rope_table_rows(start, rows, rotary_dim, base=10000.0, scaling=None, amplitude=1.0):
    """-> cos, sin [rows, rotary_dim / 2] and the angles, fp64."""
    ang = (start + np.arange(rows, dtype=np.float64))[:, None] * rope_frequencies(rotary_dim, base, scaling)
    return amplitude * np.cos(ang), amplitude * np.sin(ang), ang


def rotate_part(x, cos, sin, style):
    """x [..., D] whose first R = 2 * cos.shape[-1] dims turn by cos, sin (broadcast against x without its last axis) ->
    the rotated x, and the sum of magnitudes of each element's terms (for error bounds)."""
    x, cos, sin = to_f64(x), to_f64(cos), to_f64(sin)
    R = 2 * cos.shape[-1]
    y, size = x.copy(), np.abs(x)
    for i in range(R // 2):
        p, q = (i, i + R // 2) if style == "half" else (2 * i, 2 * i + 1)
        a, b, c, s = x[..., p], x[..., q], cos[..., i], sin[..., i]
        y[..., p], y[..., q] = a * c - b * s, b * c + a * s
        size[..., p], size[..., q] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, size


def append_paged(pages, rows, slots):
    """rows [T, Hkv, D] into pages [num_pages, Hkv, page_size, D] (numpy, in place) at their slots (-1: none)."""
    page_size = pages.shape[2]
    for t, slot in enumerate(int(s) for s in slots):
        if slot >= 0:
            pages[slot // page_size, :, slot % page_size] = rows[t]


def read_paged(pages, table_row, n):
    """Keys 0 .. n-1 of the sequence whose pages `table_row` lists, fp64 [n, Hkv, D]."""
    page_size = pages.shape[2]
    if n == 0:
        return np.zeros((0,) + (pages.shape[1], pages.shape[3]))
    return np.stack([to_f64(pages[int(table_row[j // page_size]), :, j % page_size]) for j in range(n)])


def decode_multi_paged(q, kpages, vpages, table, kv_lens, cu_new, scale):
    """q [T, Hq, D] packed by cu_new -> O [T, Hq, D], lse [T, Hq] (rows of no sequence 0 and -inf), fp64."""
    q = to_f64(q)
    T, Hq, D = q.shape
    group = Hq // kpages.shape[1]
    O, lse = np.zeros(q.shape), np.full((T, Hq), -np.inf)
    for b, n in enumerate(int(x) for x in kv_lens):
        t0, t1 = int(cu_new[b]), int(cu_new[b + 1])
        if t0 == t1 or n == 0:
            continue
        k, v = read_paged(kpages, table[b], n), read_paged(vpages, table[b], n)
        for h in range(Hq):
            O[t0:t1, h], lse[t0:t1, h] = attention_head(q[t0:t1, h], k[:, h // group], v[:, h // group], scale, causal=True)
    return O, lse


def _whole(x):
    """fp32 (or bf16) values as integers of 2^-149, exact; whatever is not finite as None."""
    x = float(x)
    return int(math.ldexp(x, 149)) if math.isfinite(x) else None


def verify_drafts(drafts, target_rows, uniforms, draft_rows=None):
    """One sequence: drafts x_0 .. x_{n-1}, target_rows [n + 1][V], uniforms [K + 1] (the last one draws the next token),
    draft_rows [n][V] or None -> (standing drafts, next token or -1)."""
    n, V = len(drafts), len(target_rows[0])
    stand = 0
    for i, x in enumerate(int(d) for d in drafts):
        if not 0 <= x < V:
            break
        p, q, u = float(target_rows[i][x]), 1.0 if draft_rows is None else float(draft_rows[i][x]), float(uniforms[i])
        if not u * q < p:  # (24-bit numbers: the product is exact in 64 bits)
            break
        stand += 1
    p = [_whole(v) for v in target_rows[stand]]
    own = [max(v, 0) if v is not None else 0 for v in p]
    w = own
    if stand < n:
        if draft_rows is None:
            w = [0 if j == int(drafts[stand]) else v for j, v in enumerate(own)]
        else:
            q = [_whole(v) for v in draft_rows[stand]]
            w = [max(a - b, 0) if a is not None and b is not None else 0 for a, b in zip(p, q)]
        if sum(w) == 0:
            w = own
    total = sum(w)
    if total == 0:
        return stand, -1
    u, last, run = float(uniforms[-1]), -1, 0
    num, den = u.as_integer_ratio() if math.isfinite(u) else (0, 0)
    for j, v in enumerate(w):
        if v > 0:
            run += v
            last = j
            if den and run * den > num * total:
                return stand, j
    return stand, last
