"""Inputs and error bounds shared by the tests of the serving-step operators."""
import numpy as np
import torch

import oracle

BF16 = 2.0 ** -8   # half a step of bf16, relative to the value
F16 = 2.0 ** -11
F32 = 2.0 ** -24


def make_pool(num_pages, Hkv, page_size, D, seed, poison=False):
    """A pool (numpy uint8) of random codes, scales and minima; with ``poison`` every pair is NaN and every code 255."""
    g = np.random.default_rng(seed)
    G = D // 64
    pool = g.integers(0, 256, (num_pages, Hkv, page_size // 16, 18 * D), dtype=np.uint8)
    pairs = np.empty(pool.shape[:3] + (2 * 16 * G, 2), np.float16)
    pairs[..., 0] = g.uniform(0.05, 0.5, pairs.shape[:-1])
    pairs[..., 1] = -7.5 * pairs[..., 0] * g.normal(1.0, 0.3, pairs.shape[:-1])
    if poison:
        pool[:] = 255
        pairs[:] = np.nan
    pool[..., 16 * D:] = pairs.reshape(pool.shape[:3] + (-1,)).view(np.uint8)
    return pool


def make_table(lens, page_size, num_pages, seed, width=None):
    """A block table of distinct random pages, -1 past each sequence's last."""
    g = np.random.default_rng(seed)
    used = [-(-n // page_size) for n in lens]
    width = width or max(1, max(used))
    perm = g.permutation(num_pages)
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, perm[at:].astype(np.int32)


def decode_bound(q, pool, table, lens, scale, out_f32):
    """Reference and error bounds of decode over the pool, q [B, Hq, Lq, D] -> O, lse, bound on O, bound on lse.

    Logits: a score is a sum of D products of an 11-bit and a 4-bit number with D/64 scalings, all in fp32; with t the
    sum of the terms' magnitudes, D/4 + 16 roundings of at most 2^-23 t cover the accumulation (whatever its order and
    whether it rounds or truncates), scaling and exponential: delta = (D/4 + 16) 2^-23 (scale t) + 2^-20.  A weight is off by
    the factor e^delta, which moves O by at most 2 delta times the sum A of p (s u + |m|) and lse by delta.  Rounding
    weights times scales to fp16 moves O by at most 2^-11 of A (two terms, fp32 output: 2^-22), sums and merges of at most 2^17
    keys in fp32 by 2^-18 of A, and the output's own rounding is BF16 (F32) of it."""
    B, Hq, Lq, D = q.shape
    Hkv = pool.shape[1]
    group = Hq // Hkv
    O, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    bO, bL = np.zeros(q.shape), np.zeros(q.shape[:3])
    q = oracle.to_f64(q)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        k, v, kt, vt = oracle.read_q4(pool, table[b], 0, n)
        for h in range(Hq):
            hk = h // group
            o, ls = oracle.attention_head(q[b, h], k[:, hk], v[:, hk], scale, causal=True)
            O[b, h], lse[b, h] = o, ls
            S = scale * q[b, h] @ k[:, hk].T
            vis = oracle.visible_mask(Lq, n, True)
            t = abs(scale) * (np.abs(q[b, h]) @ kt[:, hk].T)
            P = np.exp(np.where(vis, S, -np.inf) - np.where(np.isneginf(ls), 0.0, ls)[:, None])
            delta = (D / 4 + 16) * 2.0 ** -23 * np.where(vis, t, 0).max(-1) + 2.0 ** -20
            A = P @ vt[:, hk]
            bO[b, h] = (2 * delta[:, None] + (2.0 ** -22 if out_f32 else F16) + 2.0 ** -18) * A
            bO[b, h] += (F32 if out_f32 else BF16) * (np.abs(o) + bO[b, h])
            bL[b, h] = delta + 2.0 ** -18 + F32 * np.abs(np.where(np.isneginf(ls), 0.0, ls))
    return O, lse, bO, bL


def assert_within(x, ref, bound, what=""):
    x = x.detach().double().cpu().numpy() if isinstance(x, torch.Tensor) else np.asarray(x, np.float64)
    inf = np.isinf(ref)
    assert np.array_equal(x[inf], ref[inf]), f"{what}: infinities differ"
    d = np.abs(x - np.where(inf, 0, ref))[~inf]
    bound = np.broadcast_to(bound, ref.shape)[~inf]
    assert np.isfinite(d).all(), f"{what}: not finite"
    worst = float((d - bound).max()) if d.size else 0.0
    assert worst <= 0, f"{what}: {d[np.argmax(d - bound)]:.3e} off, bound {bound[np.argmax(d - bound)]:.3e}"
