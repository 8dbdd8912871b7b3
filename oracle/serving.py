"""Plain fp64 forms of the serving-step operators around a paged 4-bit cache -- TEST INFRASTRUCTURE ONLY.

``page_step`` is the bookkeeping, one page and one token at a time; ``qk_norm_rope`` the RMS norm of each head with
the rotation of :func:`oracle.rope_rotate`; ``quantise_q4`` / ``values_q4`` the 4-bit form of a row's groups of 64
dims; ``write_q4`` / ``read_q4`` place such rows in, and take them from, the bytes of a pool (tiles of 16 keys: K codes,
V codes, K pairs, V pairs).  Nothing here shares code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from .sdpa import to_f64

F16_MAX = 65504.0


def page_step(kv_lens, block_table, free_pages, free_count, page_size, new_lens=None, keep_lens=None):
    """-> (kv_lens, block_table, stack of free pages, slots, positions, cu_new), or None if the step is refused."""
    lens = [int(x) for x in kv_lens]
    table = [[int(x) for x in row] for row in block_table]
    stack = [int(x) for x in free_pages][:int(free_count)]
    B, width = len(lens), len(table[0])
    keep = lens if keep_lens is None else [int(x) for x in keep_lens]
    new = [0] * B if new_lens is None else [int(x) for x in new_lens]
    for a, c, n in zip(lens, keep, new):
        if not (0 <= a <= width * page_size and 0 <= c <= a and n >= 0 and c + n <= width * page_size):
            return None
    have = [-(-a // page_size) for a in lens]
    need = [-(-(c + n) // page_size) for c, n in zip(keep, new)]
    for b in reversed(range(B)):
        for i in reversed(range(need[b], have[b])):
            stack.append(table[b][i])
            table[b][i] = -1
    for b in range(B):
        for i in range(have[b], need[b]):
            if not stack:
                return None
            table[b][i] = stack.pop()
    slots, positions, cu = [], [], [0]
    for b in range(B):
        for pos in range(keep[b], keep[b] + new[b]):
            slots.append(table[b][pos // page_size] * page_size + pos % page_size)
            positions.append(pos)
        cu.append(cu[-1] + new[b])
    return [c + n for c, n in zip(keep, new)], table, stack, slots, positions, cu


def rms_norm(x, weight, eps):
    """x [..., D] times weight over the root of mean(x^2) + eps, in fp64."""
    x = to_f64(x)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * to_f64(weight)


def quantise_q4(x):
    """Groups of 64 along the last axis: x [..., D] -> codes [..., D/64, 64] (ints), scale and minimum (fp16 values as
    fp64) [..., D/64]."""
    x = np.clip(np.nan_to_num(to_f64(x), nan=0.0, posinf=F16_MAX, neginf=-F16_MAX), -F16_MAX, F16_MAX)
    x = x.reshape(*x.shape[:-1], -1, 64)
    lo, hi = x.min(-1), x.max(-1)
    m = lo.astype(np.float32).astype(np.float16).astype(np.float64)
    s = ((hi - lo) / 15).astype(np.float32).astype(np.float16).astype(np.float64)
    q = (x - m[..., None]) / np.where(s > 0, s, 1.0)[..., None]
    u = np.where((s > 0)[..., None], np.clip(np.rint(q), 0, 15), 0).astype(np.int64)
    return u, s, m


def values_q4(u, s, m):
    """scale * code + minimum, groups joined again."""
    x = u * s[..., None] + m[..., None]
    return x.reshape(*x.shape[:-2], x.shape[-2] * x.shape[-1])


def tile_parts(tile, D):
    """(codes, pairs) of K and of V in the 18 * D bytes of one tile: uint8 [G, 16, 32] and fp16 [16, G, 2], as views."""
    G = D // 64
    par = tile[16 * D:].view(np.float16)
    return ((tile[:8 * D].reshape(G, 16, 32), par[:32 * G].reshape(16, G, 2)),
            (tile[8 * D:16 * D].reshape(G, 16, 32), par[32 * G:].reshape(16, G, 2)))


def write_q4(pool, k, v, slots):
    """Rows k, v [T, Hkv, D] into their slots (-1: none) of a pool, uint8 numpy [pages, Hkv, page_size/16, 18 D]."""
    D, page_size = pool.shape[-1] // 18, 16 * pool.shape[2]
    packed = [quantise_q4(x) for x in (k, v)]
    for t, slot in enumerate(int(s) for s in slots):
        if slot < 0:
            continue
        page, off = divmod(slot, page_size)
        for h in range(pool.shape[1]):
            parts = tile_parts(pool[page, h, off // 16], D)
            for (codes, pairs), (u, s, m) in zip(parts, packed):
                codes[:, off % 16] = u[t, h, :, 0::2] | (u[t, h, :, 1::2] << 4)
                pairs[off % 16, :, 0] = s[t, h]
                pairs[off % 16, :, 1] = m[t, h]


def read_q4(pool, table_row, first, last):
    """Keys first .. last-1 of the sequence whose pages `table_row` lists: (k, v), fp64 [keys, Hkv, D], and the largest
    terms scale * code and |minimum| that make them up (same shape, for error bounds)."""
    D, page_size, Hkv = pool.shape[-1] // 18, 16 * pool.shape[2], pool.shape[1]
    G, pos = D // 64, np.arange(first, last)
    page, off = np.asarray(table_row)[pos // page_size], pos % page_size
    tiles, key = pool[page, :, off // 16], off % 16  # [keys, Hkv, 18 D]
    at = np.arange(len(pos))
    pairs = np.ascontiguousarray(tiles[..., 16 * D:]).view(np.float16).astype(np.float64)
    pairs = pairs.reshape(len(pos), Hkv, 2, 16, G, 2)
    values, terms = [], []
    for which in range(2):
        codes = tiles[..., 8 * D * which:8 * D * (which + 1)].reshape(len(pos), Hkv, G, 16, 32)[at, :, :, key]
        u = np.stack([codes & 15, codes >> 4], -1).reshape(len(pos), Hkv, G, 64)
        sm = pairs[at, :, which, key]
        values.append(values_q4(u, sm[..., 0], sm[..., 1]))
        terms.append(values_q4(u, sm[..., 0], np.abs(sm[..., 1])))
    return values[0], values[1], terms[0], terms[1]
