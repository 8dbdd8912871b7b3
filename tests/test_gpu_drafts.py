"""GPU parity of a draft step over a paged bf16 cache: rotary tables, rotated rows into pages, decode of several tokens of each
sequence over pages, verification of drafts, and a server's steps of all of them together.

Copied bits and decisions are compared for equality; computed values against fp64 with bounds counted in roundings."""
import pathlib
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from attention_attn_fwd_06_gb300 import binding as AB
from attention_attn_fwd_06_gb300.build import build
from attention_attn_fwd_06_gb300.inputs import make_decode_multi
from tests._serving import BF16, F32, assert_within, make_table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    AB.load()
    AB.attn_get_device_status()


def i32(x):
    return torch.tensor(np.asarray(x, np.int64), dtype=torch.int32, device=DEV)


def bf16(shape, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(torch.bfloat16)


def bits(t):
    return t.cpu().view(torch.int16)


# ---------------------------------------------------------------- rotary tables

SCALINGS = [None, ("linear", 4.0), ("linear", 0.3), ("base", 8.0), ("turns", 8.0, 8192, 1.0, 4.0), ("index", 32.0, 4096, 1.0, 32.0)]


@pytest.mark.parametrize("scaling", SCALINGS, ids=str)
@pytest.mark.parametrize("rows,R,start", [(1, 16, 0), (777, 48, 0), (300, 112, 1 << 20), (5000, 128, 8191), (33, 64, 2 ** 31 - 34),
                                          (100, 80, 12345)])
def test_rope_tables(rows, R, start, scaling):
    """An angle's rest (an eighth of a turn at most) is rounded to 2^-24 of itself, its sine or cosine is off by an ulp of a value
    below 1 (2^-24), the amplitude's product by 2^-24: 2^-22 in all.  The angle itself: frequencies of the library and of the
    oracle carry 2^-51 of themselves each, the oracle's product 2^-53."""
    amplitude, base = 1.3, 500000.0 if R > 64 else 10000.0
    cos, sin = AB.attn_rope_tables(rows, R, base=base, scaling=scaling, amplitude=amplitude, start=start, device=DEV)
    assert cos.shape == sin.shape == (rows, R // 2)
    c, s, ang = oracle.rope_table_rows(start, rows, R, base, scaling, amplitude)
    bound = amplitude * (2.0 ** -22 + 2.0 ** -49 * np.abs(ang))
    assert_within(cos, c, bound, "cos")
    assert_within(sin, s, bound, "sin")


def test_rope_tables_grow_and_feed_the_attention_calls():
    whole = AB.attn_rope_tables(600, 64, device=DEV)
    parts = [AB.attn_rope_tables(n, 64, start=a, device=DEV) for a, n in ((0, 1), (1, 200), (201, 399))]
    for i in range(2):
        assert torch.equal(whole[i], torch.cat([p[i] for p in parts]))
    out = torch.full((600, 32), 7.0, device=DEV), torch.full((600, 32), 7.0, device=DEV)
    got = AB.attn_rope_tables(600, 64, cos=out[0], sin=out[1])
    assert got[0] is out[0] and torch.equal(out[0], whole[0]) and torch.equal(out[1], whole[1])
    q, k, v = (bf16((1, 2, 100, 64), i).to(DEV) for i in range(3))
    o, _ = AB.attn_fwd(q, k, v, rope=(*whole, "half"))
    ref, _ = oracle.attention(q.cpu(), k.cpu(), v.cpu(), 0.125, True, rope=(whole[0].cpu(), whole[1].cpu(), "half"))
    assert np.abs(o.double().cpu().numpy() - ref).max() < 2e-2  # the prefill kernel's own bar
    assert AB.attn_rope_tables(0, 64, device=DEV)[0].shape == (0, 32)


def test_rope_tables_refusals():
    good = torch.empty(4, 32, device=DEV)
    for kw in (dict(cos=good[:, :16]), dict(cos=good.double()), dict(cos=good, sin=good.cpu()), dict(cos=good[:3])):
        with pytest.raises((ValueError, TypeError)):
            AB.attn_rope_tables(4, 64, **{"sin": good, **kw})
    for kw in (dict(base=1.0), dict(scaling=("linear", 0.0)), dict(start=-1), dict(scaling=("turns", 8.0, 4096, 4.0, 4.0))):
        with pytest.raises(AB.AttnError):
            AB.attn_rope_tables(4, 64, device=DEV, **kw)
    with pytest.raises(AB.AttnError):
        AB.attn_rope_tables(4, 24, device=DEV)


# ---------------------------------------------------------------- rows into pages

def tables(maxpos, R):
    c, s, _ = oracle.rope_table_rows(0, maxpos, R)
    return tuple(torch.from_numpy(t).float().to(DEV) for t in (c, s))


def rotated(x, rope, pos, R):
    """fp64 rotation of x [T, H, D] (bf16) and its bound: three fp32 roundings of each element's terms, then bf16's."""
    cos, sin, style = rope
    at = np.maximum(pos, 0)
    y, size = oracle.rotate_part(x, oracle.to_f64(cos.cpu())[at][:, None], oracle.to_f64(sin.cpu())[at][:, None], style)
    f = 3 * F32 * size
    b = f + BF16 * (np.abs(y) + f)
    b[..., R:] = 0  # copied
    return y, b


def place(T, page, num_pages, seed, pad=0):
    g = np.random.default_rng(seed)
    slots = g.permutation(num_pages * page)[:T].astype(np.int64)
    if pad:
        slots[T - pad:] = -1
    return slots


@pytest.mark.parametrize("T,Hq,Hkv,D,R,style,page", [
    (1, 8, 2, 128, 128, "half", 16),
    (5, 32, 8, 128, 128, "interleaved", 16),
    (9, 7, 1, 128, 96, "half", 48),          # an odd number of heads, three quarters of each
    (64, 4, 4, 64, 64, "interleaved", 1),    # pages of one key
    (33, 3, 3, 64, 16, "half", 7),           # a quarter of a head, an odd page size
    (130, 2, 2, 64, 32, "interleaved", 256),
    (70, 1, 5, 128, 16, "interleaved", 8),
    (257, 12, 3, 128, 48, "half", 64),
    (3100, 8, 8, 64, 48, "half", 16),        # runs of tokens a warp
    (7001, 4, 1, 128, 80, "interleaved", 40),
])
def test_append_paged(T, Hq, Hkv, D, R, style, page):
    g = np.random.default_rng(T + D)
    qkv = bf16((T, Hq + 2 * Hkv, D), T).to(DEV)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pad = min(3, T // 2)
    pages = -(-T // page) + 2
    slots = place(T, page, pages, T, pad)
    pos = g.integers(0, 500, T)
    if pad:
        pos[T - pad:] = -1
        slots[0] = -1  # rotated, not cached
    rope = (*tables(500, R), style)
    pools = [bf16((pages, Hkv, page, D), i).to(DEV) for i in (1, 2)]
    want = [p.clone() for p in pools]
    q_out, k_out = torch.full_like(q, 3.0), torch.full_like(k, 3.0)
    before = qkv.clone()
    got = AB.attn_kv_append_paged(k, v, *pools, i32(slots), rope=rope, positions=i32(pos), q=q, q_out=q_out, k_out=k_out)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    assert got[0] is q_out and got[1] is k_out and torch.equal(bits(qkv), bits(before))
    live = pos >= 0
    for x, y in ((q, q_out), (k, k_out)):
        ref, bound = rotated(x.cpu(), rope, pos, R)
        assert_within(y[live], ref[live], bound[live])
        assert (y[~live] == 3).all()
    # the cache holds the same bits at the slots, and everything else as it was
    keep = slots >= 0
    at = torch.from_numpy(slots[keep]).to(DEV)
    want[0][at // page, :, at % page] = k_out[torch.from_numpy(keep)]
    want[1][at // page, :, at % page] = v[torch.from_numpy(keep)]
    for a, b in zip(pools, want):
        assert torch.equal(bits(a), bits(b))
    # without the outputs that are not wanted: the same cache; in place: the same bits
    again = [bf16((pages, Hkv, page, D), i).to(DEV) for i in (1, 2)]
    assert AB.attn_kv_append_paged(k, v, *again, i32(slots), rope=rope, positions=i32(pos)) == (None, None)
    assert torch.equal(bits(again[0]), bits(pools[0])) and torch.equal(bits(again[1]), bits(pools[1]))
    AB.attn_kv_append_paged(k, v, *again, i32(slots), rope=rope, positions=i32(pos), q=q, q_out=q, k_out=k)
    mask = torch.from_numpy(live).to(DEV)
    assert torch.equal(bits(q[mask]), bits(q_out[mask])) and torch.equal(bits(k[mask]), bits(k_out[mask]))
    assert torch.equal(bits(q[~mask]), bits(before[:, :Hq][~mask])) and torch.equal(bits(again[0]), bits(pools[0]))


@pytest.mark.parametrize("D", [64, 128])
def test_append_paged_without_rotation_copies_bits(D):
    T, Hkv, page = 300, 3, 24
    raw = torch.randint(-32768, 32768, (2, T, Hkv, D), generator=torch.Generator().manual_seed(D), dtype=torch.int16).to(DEV)
    k, v = raw.view(torch.bfloat16)  # NaN payloads and infinities among them
    pages = -(-T // page)
    slots = place(T, page, pages, D)
    pools = torch.zeros(2, pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
    AB.attn_kv_append_paged(k, v, pools[0], pools[1], i32(slots))
    at = torch.from_numpy(slots).to(DEV)
    for x, pool in ((k, pools[0]), (v, pools[1])):
        assert torch.equal(bits(pool[at // page, :, at % page]), bits(x))
    pools.zero_()  # positions without a rotation: -1 leaves a token out, any other will do
    pos = torch.where(torch.arange(T) % 3 == 0, -1, 10 ** 9)
    AB.attn_kv_append_paged(k, v, pools[0], pools[1], i32(slots), positions=i32(pos))
    assert AB.attn_get_device_status() == AB.ATTN_OK
    m = (pos >= 0).to(DEV)
    for x, pool in ((k, pools[0]), (v, pools[1])):
        got = pool[at // page, :, at % page]
        assert torch.equal(bits(got[m]), bits(x[m])) and not got[~m].any()


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_append_paged_dims_that_do_not_turn_keep_their_bits(style):
    T, D, R = 40, 128, 48
    raw = torch.randint(-32768, 32768, (T, 2, D), generator=torch.Generator().manual_seed(1), dtype=torch.int16).to(DEV)
    x = raw.view(torch.bfloat16)
    pools = torch.zeros(2, T, 2, 1, D, dtype=torch.bfloat16, device=DEV)
    qo, ko = AB.attn_kv_append_paged(x, x, pools[0], pools[1], i32(range(T)), rope=(*tables(T, R), style), positions=i32(range(T)),
                                     q=x, want_k=True)
    for y in (qo, ko, pools[0][:, :, 0]):
        assert torch.equal(bits(y[..., R:].contiguous()), bits(x[..., R:].contiguous()))
    assert torch.equal(bits(pools[1][:, :, 0]), bits(x))


def test_append_paged_out_of_range_is_flagged_and_left():
    T, page = 6, 16
    k, v, q = (bf16((T, 2, 64), i).to(DEV) for i in range(3))
    rope = (*tables(10, 64), "half")
    pools = torch.zeros(2, 2, 2, page, 64, dtype=torch.bfloat16, device=DEV)
    for slots, pos, gone in (([0, 1, 32, 3, 4, 5], [0, 1, 2, 3, 4, 5], {2: "cache"}),
                             ([0, -2, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], {1: "cache"}),
                             ([0, 1, 2, 3, 4, 5], [0, 1, 2, 10, 4, 5], {3: "all"}),
                             ([0, 1, 2, 3, 4, 5], [0, 1, 2, 3, -7, 5], {4: "all"})):
        pools.zero_()
        q_out = torch.full_like(q, 3.0)
        AB.attn_kv_append_paged(k, v, pools[0], pools[1], i32(slots), rope=rope, positions=i32(pos), q=q, q_out=q_out)
        assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS
        for t in range(T):
            written = pools[1, 0, :, t].ne(0).any().item()
            assert written == (t not in gone)
            assert (q_out[t] == 3).all().item() == (gone.get(t) == "all")


def test_append_paged_offsets_past_32_bits():
    """The last pages of pools of over 2^32 bytes."""
    Hkv, page, D = 8, 256, 128
    pages = (5 << 30) // (Hkv * page * D * 2)
    pools = torch.zeros(2, pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
    k, v = (bf16((3, Hkv, D), i).to(DEV) for i in range(2))
    slots = [0, pages * page - 1, (pages - 1) * page]
    AB.attn_kv_append_paged(k, v, pools[0], pools[1], i32(slots))
    for t, s in enumerate(slots):
        assert torch.equal(pools[0][s // page, :, s % page], k[t]) and torch.equal(pools[1][s // page, :, s % page], v[t])
    assert pools[0].ne(0).any(-1).sum() == 3 * Hkv


def test_append_paged_refuses_what_it_would_misread():
    k = bf16((4, 2, 64), 0).to(DEV)
    pools = torch.zeros(2, 3, 2, 8, 64, dtype=torch.bfloat16, device=DEV)
    rope, pos = (*tables(8, 64), "half"), i32(range(4))
    ok = dict(rope=rope, positions=pos)
    for bad in (dict(q=k[:3]), dict(q_out=k), dict(k_out=k[:, :1]), dict(positions=pos[:3]), dict(positions=pos.long()),
                dict(rope=(rope[0], rope[1][:4], "half")), dict(rope=(*rope[:2], "full")), dict(q=k, q_out=k[:1].expand(4, 2, 64)),
                dict(rope=None, q=k), dict(rope=None, want_k=True)):
        with pytest.raises((ValueError, TypeError)):
            AB.attn_kv_append_paged(k, k, pools[0], pools[1], pos, **{**ok, **bad})
    for a in ((k, k[:3], pools[0], pools[1], pos), (k, k, pools[0], pools[1][:2], pos), (k, k, pools[0, 0], pools[1, 0], pos),
              (k, k, pools[0], pools[1], pos[:2]), (k.float(), k, pools[0], pools[1], pos)):
        with pytest.raises((ValueError, TypeError)):
            AB.attn_kv_append_paged(*a, **ok)
    with pytest.raises(AB.AttnError):
        AB.attn_kv_append_paged(k, k, pools[0], pools[1], pos, rope=(*tables(8, 24), "half"), positions=pos)
    with pytest.raises(AB.AttnError):
        AB.attn_kv_append_paged(k, k, pools[0], pools[1], pos, rope=rope)


# ---------------------------------------------------------------- decode over pages

def decode_bound(q, kpages, vpages, table, lens, cu, scale, f32):
    """Reference and bounds of decode over the pages, q [T, Hq, D].  A score is a sum of D products in fp32, its adds rounded or
    truncated: with t the sum of the terms' magnitudes, D/4 + 16 roundings of 2^-23 t cover it, its scaling and exponential:
    delta = (D/4 + 16) 2^-23 (scale t) + 2^-20.  A weight is off by the factor e^delta, which moves O by 2 delta times A, the
    sum of weights times |v|, and lse by delta.  Weights are rounded to bf16 before the second product (BF16 of A); its adds,
    up to 2^14 keys in 16s, truncate by 2^-23 of A each (2^-13 with the merges); the output's rounding is of its value."""
    q = oracle.to_f64(q)
    T, Hq, D = q.shape
    group = Hq // kpages.shape[1]
    O, lse = oracle.decode_multi_paged(q, kpages, vpages, table, lens, cu, scale)
    bO, bL = np.zeros(O.shape), np.zeros(lse.shape)
    for b, n in enumerate(lens):
        t0, t1 = cu[b], cu[b + 1]
        if n == 0 or t0 == t1:
            continue
        k, v = oracle.read_paged(kpages, table[b], n), oracle.read_paged(vpages, table[b], n)
        vis = oracle.visible_mask(t1 - t0, n, True)
        for h in range(Hq):
            kk, vv, qq, ls = k[:, h // group], v[:, h // group], q[t0:t1, h], lse[t0:t1, h]
            t = abs(scale) * (np.abs(qq) @ np.abs(kk).T)
            P = np.exp(np.where(vis, scale * qq @ kk.T, -np.inf) - np.where(np.isneginf(ls), 0.0, ls)[:, None])
            delta = (D / 4 + 16) * 2.0 ** -23 * np.where(vis, t, 0).max(-1) + 2.0 ** -20
            A = P @ np.abs(vv)
            e = (2 * delta[:, None] + BF16 + 2.0 ** -13) * A
            bO[t0:t1, h] = e + (F32 if f32 else BF16) * (np.abs(O[t0:t1, h]) + e)
            bL[t0:t1, h] = delta + 2.0 ** -18 + F32 * np.abs(np.where(np.isneginf(ls), 0.0, ls))
    return O, lse, bO, bL


class Cache:
    """Pages of sequences of `lens` keys; NaN wherever no key is."""

    def __init__(self, lens, Hkv, D, page, seed, width=None, spare=2):
        self.lens, self.page = list(lens), page
        num = sum(-(-n // page) for n in lens) + spare
        self.table = make_table(lens, page, num, seed, width=width)[0]
        k, v = bf16((2, num, Hkv, page, D), seed)
        used = np.zeros((num, page), bool)
        for b, n in enumerate(lens):
            for j in range(n):
                used[self.table[b][j // page], j % page] = True
        hole = torch.from_numpy(~used)[:, None, :, None]
        self.k, self.v = (x.masked_fill(hole, float("nan")) for x in (k, v))

    def on_gpu(self):
        return self.k.to(DEV), self.v.to(DEV), torch.from_numpy(self.table).to(DEV), i32(self.lens)


def check_decode(cache, new, Hq, scale=None, f32=False, seed=5, extra=0, gap=0, max_new=None, q=None):
    D = cache.k.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    cu = np.concatenate([[0], np.cumsum(new)]) + gap
    T = int(cu[-1]) + extra
    q = bf16((T, Hq, D), seed) if q is None else q
    dtype = torch.float32 if f32 else torch.bfloat16
    out, lse = torch.full((T, Hq, D), 7.0, dtype=dtype, device=DEV), torch.full((T, Hq), 7.0, device=DEV)
    AB.attn_decode_multi_paged(q.to(DEV), *cache.on_gpu(), i32(cu), max_new or max(max(new), 1), out=out, lse=lse, scale=scale,
                               out_dtype=dtype)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    assert (out[:gap] == 7).all() and (out[cu[-1]:] == 7).all() and (lse[:gap] == 7).all() and (lse[cu[-1]:] == 7).all()
    rows = slice(gap, int(cu[-1]))
    O, L, bO, bL = decode_bound(q, cache.k, cache.v, cache.table, cache.lens, [int(x) for x in cu], scale, f32)
    assert_within(out[rows], O[rows], bO[rows], "O")
    assert_within(lse[rows], L[rows], bL[rows], "lse")
    return out, lse


@pytest.mark.parametrize("lens,new,Hq,Hkv,D,page", [
    ([300, 129, 5], [4, 4, 4], 16, 4, 128, 16),
    ([256, 257, 128, 127], [8, 1, 3, 8], 32, 8, 128, 16),      # whole tiles, one past, one short
    ([200, 16], [16, 16], 8, 8, 128, 8),                       # pages of 8; exactly as many keys as tokens
    ([384, 1], [16, 1], 16, 2, 128, 128),                      # a full tile of 128 rows; a page a tile
    ([140, 77], [3, 2], 8, 2, 64, 24),                         # page ends inside a tile at other places each time
    ([1000, 640, 0, 1], [2, 0, 2, 1], 16, 4, 64, 48),          # no new tokens; no keys; one key
    ([5, 0, 64], [8, 3, 8], 8, 4, 128, 40),                    # fewer keys than tokens
    ([700, 300], [5, 4], 4, 2, 128, 256),                      # pages of two tiles
    ([700, 300], [5, 4], 4, 2, 64, 200),                       # pages longer than a tile, not whole ones
    ([513], [128], 1, 1, 64, 64),                              # 128 tokens of one head
    ([333, 90, 1], [1, 1, 1], 28, 4, 128, 32),                 # a token each, seven heads
    ([70, 80, 90], [1, 5, 2], 15, 3, 64, 72),
    ([300, 129, 5], [5, 4, 3], 32, 4, 128, 24),                # 40 rows; pages that end inside a tile
    ([640, 1, 200, 0], [3, 5, 1, 2], 48, 2, 64, 8),            # 120 rows
    ([260, 131], [16, 9], 8, 2, 128, 200),                     # 64 rows
    ([95, 33, 32, 31], [4, 1, 4, 4], 16, 4, 128, 8),           # ends around a stage of 32 keys, pages of 8
    ([191, 65, 64, 63], [4, 1, 4, 4], 32, 4, 64, 16),          # 32 rows, stages of 64 keys
    ([191, 65, 64, 63, 0], [5, 1, 4, 5, 2], 36, 4, 64, 16),    # 45 rows, a tile a warp, some tiles of no rows
    ([800, 7, 130], [8, 8, 3], 16, 2, 64, 40),                 # 64 rows
])
def test_decode_multi_paged(lens, new, Hq, Hkv, D, page):
    for f32 in (False, True):
        check_decode(Cache(lens, Hkv, D, page, sum(lens)), new, Hq, f32=f32)


def test_decode_multi_paged_rows_of_no_sequence_are_left():
    c = Cache([70, 33, 200], 2, 128, 16, 9, width=40)
    check_decode(c, [3, 0, 2], 8, gap=2, extra=4, max_new=6)
    check_decode(c, [1, 1, 1], 8, gap=1, extra=1, max_new=32)
    check_decode(c, [0, 0, 2], 8, extra=3)


@pytest.mark.parametrize("scale", [0.0, -0.2, 0.5, 3.0])
def test_decode_multi_paged_scales(scale):
    check_decode(Cache([300, 70], 2, 64, 16, 3), [3, 5], 8, scale=scale)


def test_decode_multi_paged_many_sequences():
    g = np.random.default_rng(4)
    lens = [int(x) for x in g.integers(0, 400, 75)]
    new = [int(x) for x in g.integers(0, 6, 75)]
    lens[7], new[7], lens[40], new[40] = 0, 3, 2, 5
    check_decode(Cache(lens, 2, 64, 32, 4), new, 4)


@pytest.mark.parametrize("Hq", [2, 40])
def test_decode_multi_paged_hundreds_of_sequences(Hq):
    """More sequences than the lengths kept in shared memory, most of them with nothing to do, for both kernels."""
    g = np.random.default_rng(Hq)
    lens = [int(x) for x in g.integers(0, 60, 700)]
    new = [int(x) if g.random() < 0.3 else 0 for x in g.integers(1, 4, 700)]
    lens[650], new[650], lens[699], new[699] = 500, 3, 0, 2
    check_decode(Cache(lens, 1, 64, 24, 4), new, Hq)


@pytest.mark.parametrize("D,page,Hq", [(128, 16, 4), (64, 48, 4), (128, 8, 8), (64, 32, 8), (64, 16, 9), (64, 8, 16), (128, 40, 24),
                                       (64, 128, 32)])
def test_decode_multi_paged_long_sequences_split_over_all_ctas(D, page, Hq):
    """16, 32 and more query rows; a tile whose rows one of the sequences does not have."""
    c = Cache([9000, 0, 33, 4000], 1, D, page, 6)
    a = check_decode(c, [4, 2, 3, 1], Hq)
    b = check_decode(c, [4, 2, 3, 1], Hq)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_multi_paged_peaked_logits():
    c = Cache([800, 300], 2, 128, 16, 11)
    check_decode(c, [4, 4], 8, q=bf16((8, 8, 128), 3, 6.0))


def test_decode_multi_paged_gives_the_contiguous_results():
    """Equal new tokens: attn_decode_multi on the cache that the pages describe (other tile bounds: near, not the same bits)."""
    B, Hq, Hkv, Lq, L, D, page = 3, 16, 4, 4, 600, 128, 16
    q, kc, vc, _ = make_decode_multi(B, Hq, Hkv, Lq, L, D, seed=77)
    lens = [600, 383, 17]
    want, wl = AB.attn_decode_multi(q.to(DEV), kc.to(DEV), vc.to(DEV), i32(lens), out_dtype=torch.float32)
    c = Cache(lens, Hkv, D, page, 5)
    for b, n in enumerate(lens):
        for j in range(n):
            c.k[c.table[b][j // page], :, j % page] = kc[b, :, j]
            c.v[c.table[b][j // page], :, j % page] = vc[b, :, j]
    packed = q.transpose(1, 2).reshape(B * Lq, Hq, D)
    out, lse = check_decode(c, [Lq] * B, Hq, f32=True, q=packed)
    assert (out.view(B, Lq, Hq, D).transpose(1, 2) - want).abs().max() < 2 ** -7  # two roundings of P to bf16
    assert (lse.view(B, Lq, Hq).transpose(1, 2) - wl).abs().max() < 1e-5


def test_decode_multi_paged_one_token_is_single_token_decode():
    c = Cache([700, 31, 0], 2, 64, 16, 8)
    q = bf16((3, 8, 64), 2)
    out, lse = check_decode(c, [1, 1, 1], 8, q=q)
    k, v, table, lens = c.on_gpu()
    want, wl = AB.attn_decode_paged(q.to(DEV), k, v, table, lens)
    assert (out.float() - want.float()).abs().max() < 2e-2 and torch.equal(lse[2], wl[2])
    assert (lse[:2] - wl[:2]).abs().max() < 1e-5


def test_decode_multi_paged_offsets_past_32_bits():
    """The last pages of pools of over 2^32 bytes give the bits of a small one."""
    Hkv, page, D, n = 8, 64, 128, 300
    need, got = -(-n // page), []
    big = (5 << 30) // (Hkv * page * D * 2)
    k, v = bf16((2, need, Hkv, page, D), 1).to(DEV)
    q = bf16((3, 16, D), 2).to(DEV)
    for pages in (need, big):
        pools = torch.zeros(2, pages, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
        pools[0, pages - need:], pools[1, pages - need:] = k, v
        table = torch.arange(pages - need, pages, dtype=torch.int32, device=DEV)[None]
        got.append(AB.attn_decode_multi_paged(q, pools[0], pools[1], table, i32([n]), i32([0, 3]), 3))
        del pools
    assert AB.attn_get_device_status() == AB.ATTN_OK
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_decode_multi_paged_long_cache_sampled():
    """131,072 keys of one sequence, two heads against fp64 (bounds as decode_bound's: slices of a CTA hold 1000 keys)."""
    n, page, D = 131072, 64, 128
    k, v = bf16((2, n // page, 1, page, D), 4)
    table = np.random.default_rng(1).permutation(n // page).astype(np.int32)[None]
    q = bf16((8, 4, D), 5)
    out, lse = AB.attn_decode_multi_paged(q.to(DEV), k.to(DEV), v.to(DEV), torch.from_numpy(table).to(DEV), i32([n]), i32([0, 8]), 8)
    kk, vv = (oracle.to_f64(x[torch.from_numpy(table[0]).long()].transpose(1, 2).reshape(n, D)) for x in (k, v))
    for h in (0, 3):
        qq = oracle.to_f64(q[:, h])
        O, L = oracle.attention_head(qq, kk, vv, D ** -0.5, causal=True)
        delta = (D / 4 + 16) * 2.0 ** -23 * D ** -0.5 * (np.abs(qq) @ np.abs(kk).T).max() + 2.0 ** -20
        A = np.exp(np.where(oracle.visible_mask(8, n, True), D ** -0.5 * qq @ kk.T, -np.inf) - L[:, None]) @ np.abs(vv)
        assert_within(out[:, h], O, (2 * delta + BF16 + 2.0 ** -13) * A + BF16 * np.abs(O))
        assert_within(lse[:, h], L, delta + 2.0 ** -18 + F32 * np.abs(L))


def test_decode_multi_paged_bad_lengths_pages_and_offsets_are_flagged():
    c = Cache([100, 60, 80], 2, 64, 16, 3, spare=0)
    k, v, table, lens = c.on_gpu()
    k, v = k.nan_to_num(0.0), v.nan_to_num(0.0)
    q = bf16((6, 4, 64), 1).to(DEV)
    good, gl = AB.attn_decode_multi_paged(q, k, v, table, lens, i32([0, 2, 4, 6]), 2)
    assert AB.attn_get_device_status() == AB.ATTN_OK

    def run(table=table, lens=lens, cu=(0, 2, 4, 6)):
        out = torch.full_like(good, 7.0)
        AB.attn_decode_multi_paged(q, k, v, table, lens, i32(cu), 2, out=out)
        assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS
        return out

    most = table.shape[1] * 16
    for bad, same in (([100, most + 1, 80], (0, 1, 4, 5)), ([100, -1, 80], (0, 1, 4, 5)), ([100, 2 ** 31 - 1, 80], (0, 1, 4, 5))):
        t = table.clone()
        t[1] = t[1].clamp(min=0)  # (a length past the capacity reads the whole row)
        out = run(table=t, lens=i32(bad))
        # (other shares of the same work: near, not the same bits)
        assert (out[list(same)].float() - good[list(same)].float()).abs().max() < 2 ** -6
        if bad[1] < 0:
            assert not out[2:4].any()
    for page in (-1, k.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = page
        out = run(table=t)
        assert torch.isfinite(out).all() and torch.equal(out[2:], good[2:])
    for cu, left in (((0, 3, 4, 6), [0, 1, 2]), ((0, 2, 1, 3), [2, 3, 4, 5]), ((-1, 2, 4, 6), [0, 1]), ((0, 2, 4, 7), [4, 5]),
                     ((0, 2, 2 ** 31 - 1, 4), [2, 3, 4, 5])):
        out = run(cu=cu)
        if cu != (0, 2, 1, 3):  # (there the third sequence's rows 1 and 2 are its own)
            assert (out[left] == 7).all()
        assert (out[5 if 5 not in left else 0] != 7).any() or 5 in left


@pytest.mark.parametrize("Hq", [8, 16, 80])
def test_decode_multi_paged_timeout_is_reported_and_the_next_call_is_right(monkeypatch, Hq):
    # one softmax thread of CTA 0 withholds an arrival: a bounded wait runs out after a second, the CTA winds down
    B, Hkv, page, D = 2, 8, 64, 128
    lens = [16384, 16000]
    pages = sum(-(-n // page) for n in lens)
    k, v = bf16((2, pages, Hkv, page, D), 3).to(DEV)
    table = torch.full((B, 256), -1, dtype=torch.int32)
    table[0], table[1, :250] = torch.arange(256), torch.arange(256, 506)
    args = bf16((8, Hq, D), 1).to(DEV), k, v, table.to(DEV), i32(lens), i32([0, 4, 8]), 4
    want, wl = AB.attn_decode_multi_paged(*args)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    monkeypatch.setenv("ATTN_FAULT_INJECT", "skip_arrive")
    AB.attn_decode_multi_paged(*args)
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("ATTN_FAULT_INJECT")
    out, lse = AB.attn_decode_multi_paged(*args)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_decode_multi_paged_workspaces():
    c = Cache([700, 31], 2, 64, 16, 8)
    k, v, table, lens = c.on_gpu()
    q, cu = bf16((6, 8, 64), 2).to(DEV), i32([0, 3, 6])
    want, wl = AB.attn_decode_multi_paged(q, k, v, table, lens, cu, 3)
    ws = AB.attn_decode_multi_paged_workspace(8, 2, 64, 3, device=DEV)
    for _ in range(3):  # the counters are left at zero
        out, lse = AB.attn_decode_multi_paged(q, k, v, table, lens, cu, 3, workspace=ws)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    with pytest.raises(AB.AttnError, match="SCRATCH"):
        AB.attn_decode_multi_paged(q, k, v, table, lens, cu, 3, workspace=ws[:-16])
    # one buffer for calls of few rows and of many, one after another
    big = AB.attn_decode_multi_paged_workspace(8, 2, 64, 32, device=DEV)
    long = Cache([6000, 700], 2, 64, 16, 9)
    lk = long.on_gpu()
    few = AB.attn_decode_multi_paged(q, *lk, cu, 3)
    q2, cu2 = bf16((40, 8, 64), 3).to(DEV), i32([0, 20, 40])
    many = AB.attn_decode_multi_paged(q2, *lk, cu2, 32)
    for _ in range(3):
        for args, ref in (((q, *lk, cu, 3), few), ((q2, *lk, cu2, 32), many)):
            out, lse = AB.attn_decode_multi_paged(*args, workspace=big)
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    O, L, bO, bL = decode_bound(q2.cpu(), long.k, long.v, long.table, long.lens, [0, 20, 40], 0.125, False)
    assert_within(many[0], O, bO)
    assert_within(many[1], L, bL)
    with pytest.raises((ValueError, TypeError)):
        AB.attn_decode_multi_paged(q, k, v, table, lens, cu, 3, workspace=ws.view(torch.int16))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = AB.attn_decode_multi_paged(q, k, v, table, lens, cu, 3, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_decode_multi_paged_on_several_streams_at_once():
    cases = []
    for i, (lens, new, Hq, Hkv, D, page) in enumerate([([9000], [4], 8, 2, 128, 16), ([1500, 700, 3], [3, 1, 2], 16, 16, 64, 48),
                                                       ([300] * 40, [1] * 40, 8, 2, 64, 32)]):
        c = Cache(lens, Hkv, D, page, i)
        cu = i32(np.concatenate([[0], np.cumsum(new)]))
        q = bf16((sum(new), Hq, D), i).to(DEV)
        cases.append(((q, *c.on_gpu(), cu, max(new)), AB.attn_decode_multi_paged_workspace(Hq, Hkv, D, max(new), device=DEV),
                      torch.cuda.Stream()))
    want = [AB.attn_decode_multi_paged(*a, workspace=w) for a, w, _ in cases]
    outs = [[(torch.empty_like(w[0]), torch.empty_like(w[1])) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for n in range(20):
        for (a, w, st), o in zip(cases, outs):
            AB.attn_decode_multi_paged(*a, out=o[n][0], lse=o[n][1], workspace=w, stream=st)
    torch.cuda.synchronize()
    assert AB.attn_get_device_status() == AB.ATTN_OK
    for w, got in zip(want, outs):
        assert all(torch.equal(o, w[0]) and torch.equal(ls, w[1]) for o, ls in got)


def test_decode_multi_paged_refuses_what_it_would_misread():
    c = Cache([70, 31], 2, 64, 16, 8)
    k, v, table, lens = c.on_gpu()
    q, cu = bf16((6, 8, 64), 2).to(DEV), i32([0, 3, 6])
    for a in ((q, k, v[:2], table, lens, cu, 3), (q, k, v, table[:1], lens, cu, 3), (q, k, v, table, lens, cu[:2], 3),
              (q, k, v, table.long(), lens, cu, 3), (q.float(), k, v, table, lens, cu, 3), (q, k.transpose(1, 2), v, table, lens, cu, 3),
              (q[:, ::2], k, v, table, lens, cu, 3), (q[:, :, :32], k, v, table, lens, cu, 3), (q, k, v, table, lens.cpu(), cu, 3)):
        with pytest.raises((ValueError, TypeError)):
            AB.attn_decode_multi_paged(*a)
    with pytest.raises((ValueError, TypeError)):
        AB.attn_decode_multi_paged(q, k, v, table, lens, cu, 3, out=torch.empty(5, 8, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(AB.AttnError):
        AB.attn_decode_multi_paged(q, k, v, table, lens, cu, 33)
    with pytest.raises(AB.AttnError):
        AB.attn_decode_multi_paged(q[:, :7].contiguous(), k, v, table, lens, cu, 3)


# ---------------------------------------------------------------- verification of drafts

def probabilities(rows, V, g, sharp=3.0):
    x = g.normal(size=(rows, V)) * sharp
    p = np.exp(x - x.max(-1, keepdims=True))
    return (p / p.sum(-1, keepdims=True)).astype(np.float32)


def check_verify(B, K, V, dtype=torch.float32, packed=False, point=False, seed=0, near=True, strides=False):
    g = np.random.default_rng(seed)
    n = [int(x) for x in g.integers(0, K + 1, B)]
    n[-1] = K
    q = torch.from_numpy(probabilities(max(B * K, 1), V, g).reshape(-1, V)).to(dtype)
    p = probabilities(B * (K + 1), V, g)
    if near and K:
        mix = np.repeat(q.float().numpy().reshape(B, K, V), 1, 1)
        p = p.reshape(B, K + 1, V)
        p[:, :K] = 0.7 * mix + 0.3 * p[:, :K]
    p = torch.from_numpy(p.reshape(B, K + 1, V)).to(dtype)
    q = q[:B * K].view(B, K, V)
    drafts = np.zeros((B, K), np.int64)
    for b in range(B):
        for i in range(K):
            w = q[b, i].double().numpy()
            drafts[b, i] = g.choice(V, p=w / w.sum())
    u = g.random((B, K + 1)).astype(np.float32)
    u[0, K] = 0.0
    lens = g.integers(100, 200, B)
    kw = {}
    if packed:
        rows = torch.cat([p[b, :n[b] + 1] for b in range(B)])
        kw["cu_target"] = i32(np.concatenate([[0], np.cumsum([x + 1 for x in n])]))
    else:
        rows, kw["draft_lens"] = p, i32(n)
    rows, qd = rows.to(DEV), q.to(DEV)
    if strides:  # rows within wider ones, sequences out of order
        wide = torch.zeros(*rows.shape[:-1], V + 5, dtype=dtype, device=DEV)
        wide[..., 2:V + 2] = rows
        rows = wide[..., 2:V + 2]
        qd = qd.transpose(0, 1).contiguous().transpose(0, 1)
    tokens, accepted, keep = AB.attn_verify_drafts(i32(drafts).view(B, K), rows, torch.from_numpy(u).to(DEV),
                                                   draft_probs=None if point else qd, kv_lens=i32(lens), **kw)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    for b in range(B):
        stand, token = oracle.verify_drafts(drafts[b, :n[b]], p[b].float().numpy()[:n[b] + 1], list(u[b, :n[b]]) + [u[b, K]],
                                            None if point else q[b].float().numpy()[:n[b]])
        want = list(drafts[b, :stand]) + [token] + [-1] * (K - stand)
        assert tokens[b].tolist() == want and accepted[b].item() == stand
        assert keep[b].item() == lens[b] - (n[b] - stand)
    return accepted


@pytest.mark.parametrize("B,K,V", [(1, 0, 1), (1, 1, 2), (3, 4, 7), (5, 3, 31), (2, 40, 33), (4, 5, 1000), (3, 2, 2048), (2, 3, 4099),
                                   (6, 4, 8192), (2, 2, 50001), (1, 2, 131072), (1, 1, 300004)])
@pytest.mark.parametrize("form", ["padded", "packed", "point", "strides"])
def test_verify_drafts(B, K, V, form):
    for dtype in (torch.float32, torch.bfloat16):
        check_verify(B, K, V, dtype, packed=form == "packed", point=form == "point", seed=B + V, strides=form == "strides")


def test_verify_drafts_many_sequences():
    a = check_verify(300, 6, 500, seed=3)
    assert 0 < a.float().mean() < 6
    check_verify(70, 3, 3000, seed=4, packed=True)


def run_verify(drafts, p, u, q=None, **kw):
    B, K = len(drafts), len(drafts[0])
    f = lambda x: torch.tensor(x, dtype=torch.float32, device=DEV)  # noqa: E731
    t, a, _ = AB.attn_verify_drafts(i32(drafts).view(B, K), f(p), f(u), draft_probs=None if q is None else f(q), **kw)
    return t.tolist(), a.tolist(), AB.attn_get_device_status()


def test_verify_drafts_borders_and_odd_weights():
    nan, inf = float("nan"), float("inf")
    p = [[0.5, 0.25, 0.25, 0.0], [0.0, 0.5, 0.0, 0.5]]
    q = [[0.25, 0.5, 0.25, 0.0]]
    ok = AB.ATTN_OK
    assert run_verify([[1]], [p], [[0.5, 0.9]], [q]) == ([[0, -1]], [0], ok)        # u q = p: refused
    assert run_verify([[1]], [p], [[0.49999997, 0.49999997]], [q]) == ([[1, 1]], [1], ok)
    assert run_verify([[1]], [p], [[0.0, 0.5]], [q]) == ([[1, 3]], [1], ok)         # u V = w_0 + w_1: the next one
    assert run_verify([[1]], [p], [[0.0, 1.0]], [q]) == ([[1, 3]], [1], ok)
    assert run_verify([[1]], [p], [[nan, nan]], [q]) == ([[0, -1]], [0], ok)        # NaN: refused; the last with weight
    assert run_verify([[3]], [p], [[0.5, 0.6]], [[p[0]]]) == ([[1, -1]], [0], ok)   # p nowhere above q
    assert run_verify([[0]], [[[nan, 0.25, inf, -1.0], p[1]]], [[0.5, 0.3]], [q]) == ([[1, -1]], [0], ok)
    assert run_verify([[2]], [p], [[0.25, 0.99]]) == ([[1, -1]], [0], ok)           # refused, and cannot come out
    assert run_verify([[2]], [p], [[0.24, 0.0]]) == ([[2, 1]], [1], ok)
    bad = AB.ATTN_ERR_DEVICE_BOUNDS
    assert run_verify([[1]], [[[0.0, nan, -1.0, inf]] * 2], [[0.5, 0.5]]) == ([[-1, -1]], [0], bad)
    for x in (-1, 4, 2 ** 31 - 1, -2 ** 31):  # not a token: refused; nothing is taken away, or the draft's row
        assert run_verify([[x]], [p], [[0.0, 0.7]]) == ([[1, -1]], [0], bad)
        assert run_verify([[x]], [p], [[0.0, 0.7]], [q]) == ([[0, -1]], [0], bad)


def test_verify_drafts_sums_carry_more_than_32_bits():
    """One large weight and 131,071 of 2^-26 of it: sums in 32 bits would lose them; u = 1 - 2^-24 lies well within their end."""
    V = 131072
    p = np.full((1, 1, V), 2.0 ** -26, np.float32)
    p[0, 0, 0] = 1.0
    total = 1.0 + (V - 1) * 2.0 ** -26
    for u in (1 - 2.0 ** -24, 1 - 2.0 ** -12, 0.999, 0.9980468):
        tokens, _, _ = AB.attn_verify_drafts(torch.zeros(1, 0, dtype=torch.int32, device=DEV), torch.from_numpy(p).to(DEV),
                                             torch.tensor([[u]], dtype=torch.float32, device=DEV))
        u32 = float(np.float32(u))
        want = max(0, int(np.floor((u32 * total - 1.0) * 2.0 ** 26)) + 1)
        assert tokens.item() == want


def test_verify_drafts_offsets_past_32_bits():
    """The last rows of probabilities of over 2^31 elements."""
    rows, V = 17000, 131072
    p = torch.zeros(rows, V, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(1, 2, V, dtype=torch.bfloat16, device=DEV)
    p[-3, 70000], p[-2, 5], p[-2, 131071], p[-1, 9] = 0.75, 0.25, 0.5, 1.0
    q[0, 0, 70000], q[0, 1, 5] = 0.5, 0.75
    cu, d = i32([rows - 3, rows]), i32([[70000, 5]])
    u = torch.tensor([[0.9, 0.5, 0.3]], device=DEV)
    tokens, accepted, _ = AB.attn_verify_drafts(d, p, u, draft_probs=q, cu_target=cu)
    assert tokens.tolist() == [[70000, 131071, -1]] and accepted.item() == 1  # 0.45 < 0.75; 0.375 is not below 0.25
    u[0, 1] = 0.25
    tokens, accepted, _ = AB.attn_verify_drafts(d, p, u, draft_probs=q, cu_target=cu)
    assert tokens.tolist() == [[70000, 5, 9]] and accepted.item() == 2
    assert AB.attn_get_device_status() == AB.ATTN_OK


def test_verify_drafts_lengths_and_offsets_out_of_range_are_flagged():
    p = torch.rand(3, 3, 50, device=DEV)
    u, d = torch.full((3, 3), 0.5, device=DEV), i32([[1, 2]] * 3)
    kv = i32([10, 20, 30])
    for n, clamped in (([1, 3, 2], [1, 2, 2]), ([1, -1, 2], [1, 0, 2])):
        got = AB.attn_verify_drafts(d, p, u, draft_lens=i32(n), kv_lens=kv)
        assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS
        want = AB.attn_verify_drafts(d, p, u, draft_lens=i32(clamped), kv_lens=kv)
        assert AB.attn_get_device_status() == AB.ATTN_OK and all(torch.equal(a, b) for a, b in zip(got, want))
    flat = p.view(9, 50)
    for cu, none in (([0, 3, 3, 6], 1), ([0, 3, 2, 5], 1), ([0, 3, 6, 10], 2), ([-1, 2, 4, 6], 0), ([0, 1, 5, 8], 1)):
        tokens, accepted, keep = AB.attn_verify_drafts(d, flat, u, cu_target=i32(cu), kv_lens=kv)
        status = AB.attn_get_device_status()
        assert status == (AB.ATTN_OK if cu == [0, 3, 3, 6] else AB.ATTN_ERR_DEVICE_BOUNDS)
        assert tokens[none].tolist() == [-1] * 3 and accepted[none] == 0 and keep[none] == kv[none]
        for b in range(3):
            if b != none and cu != [0, 3, 2, 5]:
                assert tokens[b, accepted[b]] >= 0


def test_verify_drafts_refuses_what_it_would_misread():
    p, u, d = torch.rand(3, 3, 50, device=DEV), torch.rand(3, 3, device=DEV), i32([[1, 2]] * 3)
    for a, kw in (((d, p[:, :2], u), {}), ((d, p, u[:, :2]), {}), ((d.long(), p, u), {}), ((d, p.double(), u), {}),
                  ((d, p.transpose(1, 2), u), {}), ((d, p, u), dict(draft_probs=p)), ((d, p, u), dict(draft_probs=p[:, :2].bfloat16())),
                  ((d, p, u), dict(cu_target=i32([0, 3, 6, 9]))), ((d, p.view(9, 50), u), dict(cu_target=i32([0, 9]))),
                  ((d, p.view(9, 50), u), dict(cu_target=i32([0, 3, 6, 9]), draft_lens=i32([1, 1, 1]))),
                  ((d, p, u), dict(keep_lens=i32([1, 2, 3]))), ((d, p, u), dict(tokens=i32([[1, 2]] * 3))), ((d, p.cpu(), u), {})):
        with pytest.raises((ValueError, TypeError)):
            AB.attn_verify_drafts(*a, **kw)


# ---------------------------------------------------------------- a server's draft steps

class Server:
    """Requests whose new tokens are packed, tokens of a fixed room (the rest is padding): a step can be captured."""

    def __init__(self, B, Hq, Hkv, D, R, style, page, room, most, V, seed=0):
        self.B, self.Hq, self.Hkv, self.D, self.R, self.most, self.room, self.V = B, Hq, Hkv, D, R, most, room, V
        width, pages = 12, 12 * B
        self.page = page
        self.lens, self.keep, self.new = i32([0] * B), i32([0] * B), i32([0] * B)
        self.table, self.free, self.count = i32([[-1] * width] * B), i32(np.random.default_rng(seed).permutation(pages)), i32([pages])
        self.slots, self.pos, self.cu = i32([0] * room), i32([0] * room), i32([0] * (B + 1))
        self.kp, self.vp = torch.full((2, pages, Hkv, page, D), float("nan"), device=DEV, dtype=torch.bfloat16)
        self.rope = (*AB.attn_rope_tables(width * page, R, scaling=("linear", 2.0), device=DEV), style)
        self.qkv = torch.zeros(room, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
        self.q = torch.zeros(room, Hq, D, dtype=torch.bfloat16, device=DEV)
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(room, Hq, device=DEV)
        self.ws = AB.attn_decode_multi_paged_workspace(Hq, Hkv, D, most, device=DEV)
        self.drafts, self.u = i32([[0] * (most - 1)] * B), torch.zeros(B, most, device=DEV)
        self.p, self.dp = torch.zeros(room, V, device=DEV), torch.zeros(B, most - 1, V, device=DEV)
        self.tokens, self.accepted = i32([[0] * most] * B), i32([0] * B)

    def step(self):
        AB.attn_page_step(self.lens, self.table, self.free, self.count, self.page, new_lens=self.new, keep_lens=self.keep,
                          slots=self.slots, positions=self.pos, cu_new=self.cu)
        x = self.qkv
        AB.attn_kv_append_paged(x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:], self.kp, self.vp, self.slots,
                                rope=self.rope, positions=self.pos, q=x[:, :self.Hq], q_out=self.q)
        AB.attn_decode_multi_paged(self.q, self.kp, self.vp, self.table, self.lens, self.cu, self.most, out=self.out, lse=self.lse,
                                   workspace=self.ws)
        # (the output head: self.p stands for its probabilities)
        AB.attn_verify_drafts(self.drafts, self.p, self.u, draft_probs=self.dp, cu_target=self.cu, kv_lens=self.lens,
                              tokens=self.tokens, accepted=self.accepted, keep_lens=self.keep)


@pytest.mark.parametrize("Hq,Hkv,D,R,style,page", [(8, 2, 128, 128, "half", 16), (4, 4, 64, 32, "interleaved", 24)])
def test_a_servers_draft_steps_in_a_graph(Hq, Hkv, D, R, style, page):
    """One captured step of all four calls and the page step, replayed: requests of ragged drafts, refused ones dropped by the
    next step, one that ends and one that takes its place; cache, outputs, tokens and lengths against the oracle each time."""
    g = np.random.default_rng(D)
    B, most, V = 5, 4, 97
    s = Server(B, Hq, Hkv, D, R, style, page, B * most + 3, most, V)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    held = [0] * B            # keys of each request that stay
    cache = [np.zeros((0, Hkv, D))] * B, [np.zeros((0, Hkv, D))] * B
    for it in range(14):
        new = [int(x) for x in g.integers(0 if it % 3 == 2 else 1, most + 1, B)]
        if it == 8:           # a request ends, another takes its row
            held[2] = 0
            keep = s.keep.tolist()
            keep[2] = 0
            s.keep.copy_(i32(keep))
        s.new.copy_(i32(new))
        s.qkv.copy_(bf16(s.qkv.shape, it))
        n = sum(new)
        probs = probabilities(s.room + B * (most - 1), V, g, 2.0)
        s.p.copy_(torch.from_numpy(probs[:s.room]))
        s.dp.copy_(torch.from_numpy(probs[s.room:]).view(B, most - 1, V))
        s.drafts.copy_(i32(g.integers(0, V, (B, most - 1))))
        s.u.copy_(torch.from_numpy(g.random((B, most)).astype(np.float32)))
        graph.replay()
        assert AB.attn_get_device_status() == AB.ATTN_OK
        lens = [h + x for h, x in zip(held, new)]
        cu = [0] + list(np.cumsum(new))
        assert s.lens.tolist() == lens and s.cu.tolist() == cu
        pos = np.concatenate([np.arange(h, h + x) for h, x in zip(held, new)]).astype(int)
        assert s.pos[:n].tolist() == pos.tolist() and (s.pos[n:] == -1).all()
        x = s.qkv[:n].cpu()
        ref, bound = rotated(x[:, :Hq], s.rope, pos, R)
        assert_within(s.q[:n], ref, bound, "q")
        kref, kb = rotated(x[:, Hq:Hq + Hkv], s.rope, pos, R)
        table, kp, vp = s.table.cpu().numpy(), s.kp.cpu(), s.vp.cpu()
        for b in range(B):
            got_k, got_v = (oracle.read_paged(t, table[b], lens[b]) for t in (kp, vp))
            assert np.array_equal(got_k[:held[b]], cache[0][b][:held[b]]) and np.array_equal(got_v[:held[b]], cache[1][b][:held[b]])
            rows = slice(cu[b], cu[b + 1])
            assert_within(got_k[held[b]:], kref[rows], kb[rows], "k")
            assert np.array_equal(got_v[held[b]:], oracle.to_f64(x[rows, Hq + Hkv:]))
            cache[0][b], cache[1][b] = got_k, got_v
        O, L, bO, bL = decode_bound(s.q[:n].cpu(), kp, vp, table, lens, cu, D ** -0.5, False)
        assert_within(s.out[:n], O, bO, "O")
        assert_within(s.lse[:n], L, bL, "lse")
        drafts, u, p, dp = s.drafts.cpu().numpy(), s.u.cpu().numpy(), s.p.cpu().numpy(), s.dp.cpu().numpy()
        for b in range(B):
            if new[b] == 0:
                assert s.tokens[b].tolist() == [-1] * most and s.keep[b] == lens[b]
                held[b] = lens[b]
                continue
            stand, token = oracle.verify_drafts(drafts[b, :new[b] - 1], p[cu[b]:cu[b + 1]], list(u[b, :new[b] - 1]) + [u[b, most - 1]],
                                                dp[b, :new[b] - 1])
            assert s.tokens[b].tolist() == list(drafts[b, :stand]) + [token] + [-1] * (most - 1 - stand)
            held[b] = lens[b] - (new[b] - 1 - stand)
            assert s.keep[b].item() == held[b]


def test_two_captured_steps_replayed_at_once():
    servers = [Server(4, 8, 2, 128, 128, "half", 16, 16, 4, 300, seed=i) for i in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in servers]
    for i, s in enumerate(servers):
        s.qkv.copy_(bf16(s.qkv.shape, i))
        s.p.copy_(torch.rand_like(s.p))
        s.new.fill_(3)
        s.dp.copy_(torch.rand_like(s.dp))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            s.step()

    def reset(s):
        s.lens.zero_(), s.keep.zero_(), s.table.fill_(-1), s.free.copy_(i32(range(48))), s.count.fill_(48)

    want = []
    for s, gr in zip(servers, graphs):
        reset(s)
        for _ in range(8):
            gr.replay()
        torch.cuda.synchronize()
        want.append([t.clone() for t in (s.out, s.lse, s.tokens, s.keep, s.lens)])
    for s in servers:
        reset(s)
    torch.cuda.synchronize()
    for _ in range(8):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert AB.attn_get_device_status() == AB.ATTN_OK
    for s, w in zip(servers, want):
        assert all(torch.equal(a, b) for a, b in zip(w, (s.out, s.lse, s.tokens, s.keep, s.lens)))


FIRST_CALLS = """
import torch
from attention_attn_fwd_06_gb300 import binding as AB
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
lens, table, free, count, new = i32([0] * 3), i32([[-1, -1]] * 3), i32(range(8)), i32([8]), i32([5, 17, 0])
slots, pos, cu = i32([0] * 22), i32([0] * 22), i32([0] * 4)
x = torch.randn(22, 8, 64, device="cuda").to(torch.bfloat16)
pages = torch.zeros(2, 8, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
cos, sin = torch.empty(2, 32, 16, device="cuda")
q, out, out2 = torch.empty(22, 4, 64, dtype=torch.bfloat16, device="cuda"), *torch.empty(2, 22, 4, 64, dtype=torch.bfloat16, device="cuda")
lse, lse2 = torch.empty(2, 22, 4, device="cuda")
ws = AB.attn_decode_multi_paged_workspace(4, 2, 64, 64)  # (a size only: nothing has run)
drafts, p, u = i32([[3] * 16] * 3), torch.rand(22, 40, device="cuda"), torch.rand(3, 17, device="cuda")
tokens, accepted, keep = i32([[0] * 17] * 3), i32([0] * 3), i32([0] * 3)

def step():
    AB.attn_rope_tables(32, 32, cos=cos, sin=sin)
    AB.attn_page_step(lens, table, free, count, 16, new_lens=new, slots=slots, positions=pos, cu_new=cu)
    AB.attn_kv_append_paged(x[:, 4:6], x[:, 6:], pages[0], pages[1], slots, (cos, sin, "half"), pos, q=x[:, :4], q_out=q)
    AB.attn_decode_multi_paged(q, pages[0], pages[1], table, lens, cu, 17, out=out, lse=lse, workspace=ws)    # 34 query rows
    AB.attn_decode_multi_paged(q, pages[0], pages[1], table, lens, cu, 64, out=out2, lse=lse2, workspace=ws)
    AB.attn_verify_drafts(drafts, p, u, cu_target=cu, kv_lens=lens, tokens=tokens, accepted=accepted, keep_lens=keep)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
state = (cos, sin, lens, table, slots, pos, cu, q, pages, out, lse, out2, lse2, tokens, accepted, keep)
got = [t.clone() for t in state]
lens.zero_(), table.fill_(-1), free.copy_(i32(range(8))), count.fill_(8), pages.zero_()
step()
assert AB.attn_get_device_status() == AB.ATTN_OK
assert all(torch.equal(a, b) for a, b in zip(got, state))
assert lens.tolist() == [5, 17, 0] and torch.isfinite(lse).all() and tokens[2].tolist() == [-1] * 17
few = [torch.empty_like(out), torch.empty_like(lse)]
cu5 = i32([0, 5, 5, 5])
status = None
try:
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        AB.attn_decode_multi_paged(q, pages[0], pages[1], table, lens, cu5, 5, out=few[0], lse=few[1])
except AB.AttnError as e:
    status = e.status  # the library's workspace is not made inside a capture
assert status == AB.ATTN_ERR_INVALID_ARG, status
AB.attn_decode_multi_paged(q, pages[0], pages[1], table, lens, cu5, 5, out=few[0], lse=few[1])
g2 = torch.cuda.CUDAGraph()
with torch.cuda.graph(g2):
    AB.attn_decode_multi_paged(q, pages[0], pages[1], table, lens, cu5, 5, out=few[0], lse=few[1])
few[0].zero_()
g2.replay()
assert (few[0][:5].float() - out[:5].float()).abs().max() < 2e-2 and AB.attn_get_device_status() == AB.ATTN_OK
"""


def test_first_calls_of_a_process_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=120,
                       cwd=pathlib.Path(__file__).parents[1])
    assert r.returncode == 0, r.stderr
