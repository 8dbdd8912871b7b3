"""GPU parity of the serving-step operators: page bookkeeping, q/k norm with rotation, the 4-bit cache's writing and
reading, decode over it, and a step of all of them together.

Page bookkeeping and the cache's bytes are compared for equality; computed values against fp64 with bounds counted
in roundings (tests/_serving.py, and beside each test)."""
import pathlib
import subprocess
import sys
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from attention_attn_fwd_06_gb300 import binding as AB
from attention_attn_fwd_06_gb300.build import build
from attention_attn_fwd_06_gb300.inputs import rope_tables
from tests._serving import BF16, assert_within, decode_bound, make_pool, make_table

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    AB.load()
    AB.attn_get_device_status()


def dev(x, dtype=None):
    x = torch.as_tensor(np.ascontiguousarray(x) if isinstance(x, np.ndarray) else x)
    return x.to(DEV, dtype) if dtype is not None else x.to(DEV)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- pages

class Pages:
    def __init__(self, B, page, width, num_pages, seed=0):
        perm = np.random.default_rng(seed).permutation(num_pages)
        self.page, self.num_pages = page, num_pages
        self.lens, self.table, self.stack = [0] * B, [[-1] * width for _ in range(B)], perm.tolist()
        self.d_lens, self.d_table = i32(self.lens), dev(np.array(self.table, np.int32))
        self.d_free, self.d_count = dev(perm.astype(np.int32)), i32([num_pages])

    def step(self, new=None, keep=None, room=None, expect=AB.ATTN_OK, offset=0):
        want = oracle.page_step(self.lens, self.table, self.stack, len(self.stack), self.page, new, keep)
        T = (sum(new) if new else 0) if room is None else room
        slots = torch.full((T + offset,), 77, dtype=torch.int32, device=DEV)[offset:]
        pos = torch.full((T,), 77, dtype=torch.int32, device=DEV)
        cu = torch.full((len(self.lens) + 1,), 77, dtype=torch.int32, device=DEV)
        AB.attn_page_step(self.d_lens, self.d_table, self.d_free, self.d_count, self.page,
                          new_lens=None if new is None else i32(new), keep_lens=None if keep is None else i32(keep),
                          slots=slots, positions=pos, cu_new=cu)
        assert AB.attn_get_device_status() == expect
        if expect != AB.ATTN_OK:
            assert (slots == -1).all() and (pos == -1).all() and (cu == 0).all()
        else:
            self.lens, self.table, self.stack, ws, wp, wc = want
            n = len(ws)
            assert slots.tolist() == ws + [-1] * (T - n) and pos.tolist() == wp + [-1] * (T - n) and cu.tolist() == wc
        assert self.d_lens.tolist() == self.lens and self.d_table.tolist() == self.table
        assert self.d_count.item() == len(self.stack) and self.d_free.tolist()[:len(self.stack)] == self.stack


@pytest.mark.parametrize("B,page,nmax", [(1, 16, 1), (3, 16, 40), (7, 48, 200), (64, 1, 5), (33, 256, 900),
                                         (300, 16, 3), (1030, 32, 2), (5000, 16, 1), (8192, 16, 1)])
def test_page_steps_in_a_row(B, page, nmax):
    g = np.random.default_rng(B + page)
    width = 4 * -(-nmax // page) + 1
    P = Pages(B, page, width, B * width + 2, seed=B)
    for step in range(4 if B > 2000 else 10):
        keep = [int(g.integers(0, a + 1)) if g.random() < 0.3 else a for a in P.lens] if step % 3 else None
        left = [width * page - a for a in (keep or P.lens)]
        new = [min(int(g.integers(0, nmax + 1)), x) for x in left] if step % 4 != 3 else None
        P.step(new, keep, room=(sum(new) if new else 0) + (step % 2) * 5, offset=step % 3)
    P.step(keep=[0] * B)  # everything given back
    assert sorted(P.stack) == list(range(P.num_pages))


def test_page_step_prompts_of_many_tokens():
    P = Pages(5, 16, 1100, 4000, seed=3)
    P.step(new=[17000, 0, 1, 9001, 12345])  # lists long enough for the cluster of CTAs
    P.step(new=[1, 1, 1, 1, 1], room=8)
    P.step(new=[0, 8000, 3, 0, 5000], keep=[0, 1, 2, 100, 0], room=16384)
    P.step(keep=[0] * 5)


def test_page_step_refusals_leave_everything():
    P = Pages(2, 16, 4, 5, seed=1)
    P.step(new=[33, 16])
    P.step(new=[0, 17], expect=AB.ATTN_ERR_DEVICE_POOL)              # 1 page left, 2 wanted
    P.step(new=[0, 17], keep=[10, 16])                               # row 0 gives two back first
    P.step(new=[64, 0], expect=AB.ATTN_ERR_DEVICE_BOUNDS)            # 10 + 64 keys: five pages
    P.step(new=[-1, 0], room=4, expect=AB.ATTN_ERR_DEVICE_BOUNDS)
    P.step(new=[2, 2], keep=[11, 33], expect=AB.ATTN_ERR_DEVICE_BOUNDS)   # 11 of 10 kept
    P.step(new=[2, 2], keep=[-1, 33], expect=AB.ATTN_ERR_DEVICE_BOUNDS)
    P.step(new=[2, 2], room=3, expect=AB.ATTN_ERR_DEVICE_BOUNDS)     # four tokens, room for three
    P.step(new=[2 ** 31 - 1, 2 ** 31 - 1], room=3, expect=AB.ATTN_ERR_DEVICE_BOUNDS)
    P.d_count.fill_(9)                                               # more free pages than pages
    P.stack = P.stack + [0] * (9 - len(P.stack))
    slots = i32([5, 5])
    AB.attn_page_step(P.d_lens, P.d_table, P.d_free, P.d_count, 16, new_lens=i32([1, 1]), slots=slots)
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS and slots.tolist() == [-1, -1]


@pytest.mark.parametrize("rows", [[2 ** 30 - 1] * 8, [2 ** 30 - 1, 2 ** 30 - 1, 2], [2 ** 30] * 4, [0, 2 ** 30 - 1, 0, 2 ** 30 - 1] * 9])
def test_page_step_token_sums_past_32_bits_are_refused(rows):
    # every row's length is allowed, the sum is 2^31 or more (of two, four and more rows: 0 modulo 2^32 among them)
    B, pages = len(rows), 1 << 20
    lens, table, new = i32([0] * B), torch.full((B, pages), -1, dtype=torch.int32, device=DEV), i32(rows)
    free, count, cu = i32(range(64)), i32([64]), i32([7] * (B + 1))
    AB.attn_page_step(lens, table, free, count, 1024, new_lens=new, cu_new=cu)
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS
    assert lens.tolist() == [0] * B and count.item() == 64 and cu.tolist() == [0] * (B + 1) and (table == -1).all()


def test_page_step_lists_without_room():
    """An empty list is a list: tokens it has no room for are refused, a step without tokens is not."""
    for name in ("slots", "positions"):
        P = Pages(2, 16, 4, 8, seed=1)
        empty = {name: torch.empty(0, dtype=torch.int32, device=DEV)}
        AB.attn_page_step(P.d_lens, P.d_table, P.d_free, P.d_count, 16, new_lens=i32([1, 0]), **empty)
        assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS
        assert P.d_lens.tolist() == [0, 0] and P.d_count.item() == 8
        AB.attn_page_step(P.d_lens, P.d_table, P.d_free, P.d_count, 16, new_lens=i32([0, 0]), **empty)
        assert AB.attn_get_device_status() == AB.ATTN_OK and P.d_lens.tolist() == [0, 0]


def test_page_step_bad_page_ids_are_flagged():
    P = Pages(1, 16, 4, 4, seed=2)
    P.step(new=[20])
    P.d_table[0, 1] = 9  # the page that token 20 lands on
    slots = i32([5])
    AB.attn_page_step(P.d_lens, P.d_table, P.d_free, P.d_count, 16, new_lens=i32([1]), slots=slots)
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS and slots.tolist() == [-1]
    assert P.d_lens.tolist() == [21]
    AB.attn_page_step(P.d_lens, P.d_table, P.d_free, P.d_count, 16, keep_lens=i32([16]))  # and when it goes back
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS and P.d_lens.tolist() == [16]
    AB.attn_page_step(P.d_lens, P.d_table, P.d_free, P.d_count, 16, new_lens=i32([1]), slots=slots)  # and is taken
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS and slots.tolist() == [-1]


def test_page_step_without_lists():
    P = Pages(3, 16, 4, 12, seed=5)
    AB.attn_page_step(P.d_lens, P.d_table, P.d_free, P.d_count, 16, new_lens=i32([5, 40, 0]))
    assert P.d_lens.tolist() == [5, 40, 0] and P.d_count.item() == 12 - 4
    assert AB.attn_get_device_status() == AB.ATTN_OK


# ---------------------------------------------------------------- norm and rotation

def norm_ref(x, w, pos, rope, eps, valid):
    """x [T, H, D] -> reference and bound.  An output is y_a c - y_b s with y within 2^-21 of its own size (a fp32
    sum of squares of D <= 128 terms, a reciprocal root good to 2^-22, two products): 2^-20 of the pair's size, then one
    rounding to bf16."""
    y = oracle.rms_norm(x, w, eps)
    D = x.shape[-1]
    ref, size = y.copy(), np.abs(y)
    if rope is not None:
        cos, sin, style = rope
        ref = np.stack([oracle.rope_rotate(y[:, h], np.maximum(pos, 0), cos.cpu().numpy(), sin.cpu().numpy(), style)
                        for h in range(x.shape[1])], 1)
        pair = (np.arange(D) + D // 2) % D if style == "half" else np.arange(D) ^ 1
        size = size + size[..., pair]
    ref = np.where(valid[:, None, None], ref, 7.0)
    bound = np.where(valid[:, None, None], BF16 * np.abs(ref) + 2.0 ** -19 * size + 1e-30, 0.0)
    return ref, bound


@pytest.mark.parametrize("T,Hq,Hkv,D,style", [
    (1, 1, 1, 128, "half"), (1, 32, 8, 128, "half"), (8, 32, 8, 128, "interleaved"), (3, 5, 1, 64, "half"),
    (67, 28, 4, 128, "half"), (130, 16, 16, 64, "interleaved"), (2000, 7, 7, 64, "half"), (4100, 32, 8, 128, "half"),
    (9, 4, 2, 128, None), (9, 3, 0, 64, None), (50, 6, 0, 128, "interleaved"),
])
@pytest.mark.parametrize("weights", [True, False])
def test_qk_norm_rope(T, Hq, Hkv, D, style, weights):
    g = torch.Generator().manual_seed(T + Hq)
    qkv = torch.randn(T, Hq + 2 * Hkv + 1, D, generator=g) * torch.exp(2 * torch.randn(T, 1, 1, generator=g))
    qkv[0, 0] = 0  # a row of zeros: eps alone
    qkv = dev(qkv.to(torch.bfloat16))
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv] if Hkv else None
    wq, wk = (dev((1 + torch.randn(2, D, generator=g)).to(torch.bfloat16))) if weights else (None, None)
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32)
    if T > 2:
        pos[T // 2] = -1  # a padded row among them
    valid = (pos >= 0).numpy()
    rope = None if style is None else tuple(x.to(DEV) for x in rope_tables(500, D)) + (style,)
    qo = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((T, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) if Hkv else None
    AB.attn_qk_norm_rope(q, k, wq, wk if Hkv else None, rope, dev(pos), eps=1e-5, q_out=qo, k_out=ko)
    for x, w, out in ((q, wq, qo), (k, wk, ko)):
        if x is not None:
            ref, bound = norm_ref(oracle.to_f64(x), w, pos.numpy(), rope, 1e-5, valid)
            assert_within(out, ref, bound)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    # in place, over the views of the projection: the same bits, the rest untouched
    before = qkv.clone()
    AB.attn_qk_norm_rope(q, k, wq, wk if Hkv else None, rope, dev(pos), eps=1e-5, q_out=q, k_out=k)
    assert torch.equal(q[valid], qo[valid]) and torch.equal(q[~valid], before[:, :Hq][~valid])
    if Hkv:
        assert torch.equal(k[valid], ko[valid])
    assert torch.equal(qkv[:, Hq + Hkv:], before[:, Hq + Hkv:])


def long_norm_case(T, Hq, Hkv, D, style, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(T, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    k = torch.randn(T, Hkv, D, generator=g, device=DEV).to(torch.bfloat16)
    pos = torch.randint(0, 3000, (T,), generator=g, device=DEV, dtype=torch.int32)
    pos[torch.rand(T, generator=g, device=DEV) < 0.1] = -1  # padded rows inside the warps' runs of tokens
    pos[T // 3:T // 3 + 70] = -1
    return q, k, pos, tuple(x.to(DEV) for x in rope_tables(3000, D)) + (style,)


@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (9, 2)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_qk_norm_rope_runs_of_tokens(style, D, Hq, Hkv):
    """About seven tokens a warp: the buffers of table rows are refilled, with one round of heads a token and with several."""
    q, k, pos, rope = long_norm_case(20011, Hq, Hkv, D, style, D)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    AB.attn_qk_norm_rope(q, k, None, None, rope, pos, eps=1e-5, q_out=qo, k_out=ko)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    p = pos.cpu().numpy()
    for x, out in ((q, qo), (k, ko)):
        ref, bound = norm_ref(oracle.to_f64(x.cpu()), None, p, rope, 1e-5, p >= 0)
        assert_within(out, ref, bound)


@pytest.mark.parametrize("T,Hq,Hkv,D,style", [(70001, 32, 8, 128, "half"), (130003, 2, 1, 64, "interleaved"),
                                              (130003, 5, 4, 128, "half"), (130003, 16, 2, 64, "half"),
                                              (200000, 1, 1, 128, "interleaved")])
def test_qk_norm_rope_longest_runs(T, Hq, Hkv, D, style):
    """Tens of tokens a warp, and past 32 more warps instead: the bits of calls of a token a warp over parts of it."""
    q, k, pos, rope = long_norm_case(T, Hq, Hkv, D, style, T)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    AB.attn_qk_norm_rope(q, k, None, None, rope, pos, q_out=qo, k_out=ko)
    qs, ks = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    for t in range(0, T, 2000):
        at = slice(t, min(T, t + 2000))
        AB.attn_qk_norm_rope(q[at], k[at], None, None, rope, pos[at].contiguous(), q_out=qs[at], k_out=ks[at])
    assert AB.attn_get_device_status() == AB.ATTN_OK
    assert torch.equal(qo, qs) and torch.equal(ko, ks)


@pytest.mark.parametrize("D", [64, 128])
def test_qk_norm_rope_dense_layout(D):
    B, Hq, Hkv, L = 3, 6, 2, 37
    q = dev(torch.randn(B, Hq, L, D).to(torch.bfloat16))
    k = dev(torch.randn(B, L, Hkv, D).to(torch.bfloat16)).transpose(1, 2)  # [B, H, L, D] of other strides
    rope = tuple(x.to(DEV) for x in rope_tables(64, D)) + ("half",)
    pos = dev(torch.arange(L, dtype=torch.int32).repeat(B, 1) + torch.tensor([[0], [5], [27]], dtype=torch.int32))
    qo, ko = AB.attn_qk_norm_rope(q, k, None, None, rope, pos)
    p = pos.cpu().numpy().reshape(-1)
    for x, out in ((q, qo), (k, ko)):
        flat = x.transpose(1, 2).reshape(B * L, -1, D)
        ref, bound = norm_ref(oracle.to_f64(flat), None, p, rope, 1e-6, np.ones(B * L, bool))
        assert_within(out.transpose(1, 2).reshape(B * L, -1, D), ref, bound)


def test_one_token_of_any_stride():
    """A single token's (head's) row may come with any stride: the same bits as from a contiguous tensor."""
    g = torch.Generator().manual_seed(1)
    q, k = dev(torch.randn(1, 4, 64, generator=g).to(torch.bfloat16)), dev(torch.randn(1, 1, 64, generator=g).to(torch.bfloat16))
    odd_q, odd_k = q.as_strided(q.shape, (3, 64, 1)), k.as_strided(k.shape, (1, 5, 1))
    want, got = AB.attn_qk_norm_rope(q, k), AB.attn_qk_norm_rope(odd_q, odd_k)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    out = torch.empty_like(q), torch.empty_like(k)
    AB.attn_qk_norm_rope(q, k, q_out=out[0].as_strided(q.shape, (3, 64, 1)), k_out=out[1].as_strided(k.shape, (1, 5, 1)))
    assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])
    pools = [AB.attn_kv_q4_pool(1, 1, 16, 64, DEV) for _ in range(2)]
    AB.attn_kv_append_q4(k, k, pools[0], i32([5]))
    AB.attn_kv_append_q4(odd_k, odd_k, pools[1], i32([5]))
    assert torch.equal(*pools) and AB.attn_get_device_status() == AB.ATTN_OK


def test_qk_norm_rope_refuses_what_it_would_misread():
    q = dev(torch.randn(4, 2, 64).to(torch.bfloat16))
    cos = torch.zeros(8, 32, device=DEV)
    for rope in ((cos[:0], cos[:0], "half"), (cos, cos[:4], "half"), (cos, cos.double(), "half"), (cos, cos, "both"),
                 (cos, cos, "half", q)):
        with pytest.raises((ValueError, TypeError)):
            AB.attn_qk_norm_rope(q, None, rope=rope, positions=i32([0, 1, 2, 3]))
    with pytest.raises(ValueError):
        AB.attn_qk_norm_rope(q, None, positions=i32([0, 1, 2]))
    with pytest.raises(ValueError):
        AB.attn_qk_norm_rope(q, q[:3])
    with pytest.raises(ValueError, match="overlap"):
        AB.attn_qk_norm_rope(q, None, q_out=q[:1].expand(4, 2, 64))
    with pytest.raises(AB.AttnError) as e:  # a view that does not start on 16 bytes
        AB.attn_qk_norm_rope(torch.zeros(4 * 128 + 4, dtype=torch.bfloat16, device=DEV)[4:].view(4, 2, 64), None)
    assert e.value.status == AB.ATTN_ERR_ALIGNMENT
    with pytest.raises(AB.AttnError) as e:  # rotation without positions
        AB.attn_qk_norm_rope(q, None, rope=(cos, cos, "half"))
    assert e.value.status == AB.ATTN_ERR_INVALID_ARG


def test_qk_norm_rope_positions_out_of_range_are_flagged():
    q = dev(torch.randn(4, 2, 64).to(torch.bfloat16))
    rope = tuple(x.to(DEV) for x in rope_tables(10, 64)) + ("half",)
    out = torch.full_like(q, 7.0)
    AB.attn_qk_norm_rope(q, None, rope=rope, positions=i32([9, 10, -2, -1]), q_out=out)
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS
    assert (out[1:] == 7).all() and not (out[0] == 7).any()


# ---------------------------------------------------------------- the 4-bit cache

@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 64, 16), (1, 8, 128, 16), (5, 3, 128, 48), (130, 4, 64, 256),
                                          (1000, 2, 128, 32), (333, 16, 64, 16)])
def test_append_writes_the_oracle_bytes(T, Hkv, D, page):
    g = torch.Generator().manual_seed(T)
    num_pages = -(-T // page) + 3
    x = torch.randn(T, 2 * Hkv + 1, D, generator=g) * torch.exp(2 * torch.randn(1, 2 * Hkv + 1, D, generator=g))
    x[0, 0, :64] = 2.5                       # a group of one value
    x[0, Hkv, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1e30])
    x[-1, 0] = 0
    x[-1, -2] *= 1e-9                        # scales below fp16's range
    x = x.to(torch.bfloat16)
    k, v = x[:, :Hkv], x[:, Hkv:2 * Hkv]
    slots = torch.randperm(num_pages * page, generator=g)[:T].to(torch.int32)
    if T > 3:
        slots[2] = -1
    pool = make_pool(num_pages, Hkv, page, D, 1, poison=True)
    got = dev(pool.copy())
    xd = dev(x)
    AB.attn_kv_append_q4(xd[:, :Hkv], xd[:, Hkv:2 * Hkv], got, dev(slots))
    oracle.write_q4(pool, k, v, slots)
    assert np.array_equal(got.cpu().numpy(), pool)
    assert AB.attn_get_device_status() == AB.ATTN_OK


def test_append_ties_and_borders_match_exact_decisions():
    # Values on and one bf16 step beside the middle between two codes: extremes 0 and 15 s make the scale s exactly.
    rows = []
    for s in (1.0, 2.0 ** -5, 3.0, 0.34375):
        mid = (torch.arange(15, dtype=torch.float64) + 0.5) * s
        x = torch.zeros(64, dtype=torch.float64)
        x[1] = 15 * s
        x[2:17], x[17:32], x[32:47] = mid, mid * (1 + 2.0 ** -8), mid * (1 - 2.0 ** -8)
        rows.append(x)
    k = torch.stack(rows)[:, None].to(torch.bfloat16)
    for off in (0.0, -7.0, 100.0):
        kk = (k.double() + off).to(torch.bfloat16)
        pool = make_pool(1, 1, 16, 64, 1)
        got = dev(pool.copy())
        AB.attn_kv_append_q4(dev(kk), dev(kk), got, i32(range(4)))
        oracle.write_q4(pool, kk, kk, range(4))
        assert np.array_equal(got.cpu().numpy(), pool)


def test_append_values_a_hair_beside_a_border():
    """x - minimum is a border between two codes but for a part too small for fp32: by the definition that part decides.
    Expected codes by rational arithmetic."""
    rows = []
    for s, k in ((1.0, 0), (1.0, 1), (2.0 ** -3, 6), (2.0 ** -3, 7), (3.0, 10), (0.34375, 13), (2.0 ** -5, 14)):
        border = (k + 0.5) * s
        x = torch.zeros(64, dtype=torch.float64)  # small values over a minimum of minus the border, 0 among them
        x[0], x[1] = -border, 15 * s - border
        x[2:34] = 2.0 ** -torch.arange(18, 50, dtype=torch.float64) * border
        x[34:60] = -(2.0 ** -torch.arange(18, 122, 4, dtype=torch.float64)) * border
        x[60] = 2.0 ** -126
        rows.append(x)
        for m in (2.0 ** -24, -(2.0 ** -24), 3 * 2.0 ** -20, -(2.0 ** -14), -(2.0 ** -9)):
            x = torch.full((64,), border, dtype=torch.float64)  # the border over a small minimum
            x[0], x[1], x[2] = m, 15 * s, border * (1 + 2.0 ** -7)
            rows.append(x)
    k = torch.stack(rows)[:, None].to(torch.bfloat16)
    T = k.shape[0]
    assert T <= 48
    pool = AB.attn_kv_q4_pool(3, 1, 16, 64, DEV)
    AB.attn_kv_append_q4(dev(k), dev(k), pool, i32(range(T)))
    assert AB.attn_get_device_status() == AB.ATTN_OK
    _, s, m = oracle.quantise_q4(k)
    got, seen = pool.cpu().numpy(), 0
    for t in range(T):
        scale, least = Fraction(float(s[t, 0, 0])), Fraction(float(m[t, 0, 0]))
        want = [min(15, max(0, round((Fraction(float(x)) - least) / scale))) for x in k[t, 0].double()]  # ties to even
        seen += sum(u != min(15, max(0, round(float(np.float32(x) - np.float32(least)) / float(scale))))
                    for u, x in zip(want, k[t, 0].float().numpy()))
        for codes, pairs in oracle.serving.tile_parts(got[t // 16, 0, 0], 64):
            u = np.stack([codes[0, t % 16] & 15, codes[0, t % 16] >> 4], -1).reshape(-1)
            assert pairs[t % 16, 0].tolist() == [float(scale), float(least)] and u.tolist() == want, t
    assert seen > 100  # values that fp32's difference would put on the border


def test_append_slots_out_of_the_pool_are_flagged():
    k = dev(torch.randn(3, 2, 64).to(torch.bfloat16))
    pool = dev(make_pool(2, 2, 16, 64, 1))
    before = pool.clone()
    AB.attn_kv_append_q4(k, k, pool, i32([32, -7, -1]))
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS and torch.equal(pool, before)


@pytest.mark.parametrize("B,Hkv,D,page,hi", [(1, 1, 64, 16, 1), (4, 8, 128, 16, 100), (3, 3, 128, 48, 300),
                                             (9, 2, 64, 256, 700), (70, 4, 64, 32, 50)])
def test_gather_reads_the_oracle_values(B, Hkv, D, page, hi):
    g = np.random.default_rng(B)
    lens = [int(x) for x in g.integers(0, hi + 1, B)]
    lens[-1] = hi
    starts = [int(g.integers(0, n + 1)) if b % 2 else 0 for b, n in enumerate(lens)]
    num_pages = sum(-(-n // page) for n in lens) + 2
    pool = make_pool(num_pages, Hkv, page, D, 2)
    table, _ = make_table(lens, page, num_pages, 3)
    cu = np.concatenate([[0], np.cumsum([n - s for n, s in zip(lens, starts)])])
    total = int(cu[-1]) + 5  # rows behind the last sequence
    ko, vo = (torch.full((total, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    AB.attn_kv_gather_q4(dev(pool), dev(table), i32(cu), total, kv_starts=i32(starts), k_out=ko, v_out=vo)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    parts = [oracle.read_q4(pool, table[b], starts[b], lens[b])[:2] for b in range(B)]
    for i, out in enumerate((ko, vo)):
        ref = torch.from_numpy(np.concatenate([p[i] for p in parts])).float().to(torch.bfloat16)  # s u exact in fp32
        assert torch.equal(out.cpu()[:int(cu[-1])], ref) and (out[int(cu[-1]):] == 7).all()


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_start_on_16_bytes(D):
    """The same bytes whether rows start on 32 bytes or only on 16: by their base, by a stride, and on the way back."""
    T, Hkv, page = 45, 3, 16
    x = dev(torch.randn(2, T, Hkv, D, generator=torch.Generator().manual_seed(D)).to(torch.bfloat16))
    slots, table, cu = i32(range(T)), i32(range(3))[None], i32([0, T])

    def shifted(rows=None):
        t = torch.empty(T * Hkv * D + 8, dtype=torch.bfloat16, device=DEV)[8:].view(T, Hkv, D)
        return t if rows is None else t.copy_(rows)

    def strided(rows):
        return torch.empty(T, Hkv, D + 8, dtype=torch.bfloat16, device=DEV)[..., :D].copy_(rows)

    pools = []
    for k, v in ((x[0], x[1]), (shifted(x[0]), x[1]), (x[0], shifted(x[1])), (strided(x[0]), x[1]), (x[0], strided(x[1]))):
        pools.append(AB.attn_kv_q4_pool(3, Hkv, page, D, DEV))
        AB.attn_kv_append_q4(k, v, pools[-1], slots)
    assert all(torch.equal(p, pools[0]) for p in pools)
    want = AB.attn_kv_gather_q4(pools[0], table, cu, T)
    for k, v in ((shifted(), None), (None, shifted())):
        got = AB.attn_kv_gather_q4(pools[0], table, cu, T, k_out=k, v_out=v)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert AB.attn_get_device_status() == AB.ATTN_OK


def test_gather_out_of_range_rows_are_flagged_and_left():
    pool = dev(make_pool(3, 1, 16, 64, 2))
    for table, start in (([[0, 7]], 0), ([[0, -1]], 0), ([[0, 1]], 20), ([[0, 1]], -3)):
        ko, vo = AB.attn_kv_gather_q4(pool, i32(table[0])[None], i32([0, 32]), 32, kv_starts=i32([start]),
                                      k_out=torch.full((32, 1, 64), 7.0, dtype=torch.bfloat16, device=DEV))
        assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS
        bad = {0: slice(16, 32), 20: slice(12, 32), -3: slice(0, 3)}[start]
        good = {0: slice(0, 16), 20: slice(0, 12), -3: slice(3, 32)}[start]
        assert (ko[bad] == 7).all() and not (ko[good] == 7).all(-1).any()


# ---------------------------------------------------------------- decode

def run_decode(q, pool, table, lens, scale, **kw):
    out, lse = AB.attn_decode_q4(dev(q), dev(pool), dev(table), i32(lens), scale=scale, **kw)
    torch.cuda.synchronize()
    assert AB.attn_get_device_status() == AB.ATTN_OK
    return out, lse


def check_decode(B, Hq, Hkv, Lq, D, page, lens, seed=0, scale=None, chunks=(0,), qscale=1.0, poison_rest=True):
    g = torch.Generator().manual_seed(seed)
    num_pages = sum(-(-n // page) for n in lens) + 2
    pool = make_pool(num_pages, Hkv, page, D, seed)
    table, _ = make_table(lens, page, num_pages, seed + 1)
    if poison_rest:  # what no key holds is NaN: pages of nobody, and the rows behind each last key
        held = set()
        bad = make_pool(1, Hkv, page, D, 0, poison=True)[0]
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                held.add(int(table[b, i]))
                for off in range(max(0, n - i * page), page):
                    for h in range(Hkv):
                        for (c, p), (cb, pb) in zip(oracle.serving.tile_parts(pool[table[b, i], h, off // 16], D),
                                                    oracle.serving.tile_parts(bad[h, off // 16], D)):
                            c[:, off % 16], p[off % 16] = cb[:, off % 16], pb[off % 16]
        for i in set(range(num_pages)) - held:
            pool[i] = bad
    q = (torch.randn(B, Hq, Lq, D, generator=g) * qscale).to(torch.bfloat16)
    scale = D ** -0.5 if scale is None else scale
    qq = q if Lq > 1 else q[:, :, 0].contiguous()
    for f32 in (False, True):
        O, lse, bO, bL = decode_bound(q, pool, table, lens, scale, f32)
        for chunk in chunks:
            out, ls = run_decode(qq, pool, table, lens, scale, chunk=chunk,
                                 out_dtype=torch.float32 if f32 else torch.bfloat16)
            assert_within(out.view(q.shape), O, bO, f"O f32={f32} chunk={chunk}")
            assert_within(ls.view(q.shape[:3]), lse, bL, f"lse f32={f32} chunk={chunk}")


@pytest.mark.parametrize("B,Hq,Hkv,Lq,D,page,lens", [
    (1, 1, 1, 1, 64, 16, [1]),
    (1, 1, 1, 1, 128, 16, [16]),
    (2, 4, 4, 1, 128, 16, [300, 17]),
    (3, 16, 4, 1, 128, 48, [513, 64, 65]),
    (2, 16, 2, 1, 128, 64, [257, 128]),     # 8 heads per kv head
    (1, 32, 2, 1, 128, 16, [130]),          # 16: two column groups in one CTA
    (1, 40, 2, 1, 64, 32, [200]),           # 20: two row chunks
    (2, 12, 4, 1, 128, 16, [100, 3]),       # 3
    (2, 14, 2, 1, 64, 256, [333, 129]),     # 7
    (4, 8, 2, 1, 64, 16, [0, 1, 0, 90]),    # empty sequences among them
    (2, 8, 2, 3, 128, 16, [50, 2]),         # 3 tokens, one sequence of 2 keys: a token that sees none
    (2, 8, 2, 8, 128, 32, [300, 9]),        # 32 query rows
    (1, 32, 8, 5, 64, 16, [77]),            # 20 query rows
    (1, 4, 1, 32, 128, 48, [200]),          # 128
    (2, 6, 2, 2, 64, 16, [1, 640]),
])
def test_decode_q4(B, Hq, Hkv, Lq, D, page, lens):
    check_decode(B, Hq, Hkv, Lq, D, page, lens, seed=sum(lens), chunks=(0, 1, 100))


@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_decode_q4_scales(scale):
    check_decode(2, 8, 2, 1, 128, 16, [190, 33], seed=5, scale=scale)


@pytest.mark.parametrize("qscale", [1e-20, 1e-3, 30.0, 1e4])
def test_decode_q4_query_magnitudes(qscale):
    check_decode(1, 8, 2, 1, 128, 16, [150], seed=6, qscale=qscale, scale=0.09 / max(qscale, 1.0))


def test_decode_q4_values_of_unlike_sizes():
    # Scales of V that grow a thousandfold from key to key and shrink to subnormals: the weights' common factor follows.
    D, page, n = 128, 16, 160
    pool = make_pool(12, 1, page, D, 9)
    table, _ = make_table([n], page, 12, 9)
    for pos in range(n):
        _, (codes, pairs) = oracle.serving.tile_parts(pool[table[0, pos // page], 0, 0], D)
        f = [1e-7, 1e-4, 1.0, 50.0, 900.0][pos // 32]
        pairs[pos % 16] = (pairs[pos % 16].astype(np.float64) * f).astype(np.float16)
    q = torch.randn(1, 4, 1, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for lens in ([n], [32], [64]):
        for f32 in (False, True):
            O, lse, bO, bL = decode_bound(q, pool, table, lens, 0.05, f32)
            out, ls = run_decode(q[:, :, 0].contiguous(), pool, table, lens, 0.05, chunk=1 << 20,
                                 out_dtype=torch.float32 if f32 else torch.bfloat16)
            assert_within(out[:, :, None], O, bO)
            assert_within(ls[:, :, None], lse, bL)


def check_first_key_leads(n, D, Hq, scales, types, odd_key=None, odd_scale=None):
    """A row in one slice whose first key's weight is 2^21 times the others', V's scales drawn from an interval; one other
    key may have a scale of its own, and a logit 60 below the rest if that scale is large."""
    g, page = np.random.default_rng(n), 64
    num = n // page
    pool = make_pool(num, 1, page, D, 3)
    pairs = np.empty((num, 1, page // 16, 2, 16, D // 64, 2), np.float16)
    k, v = np.moveaxis(pairs, 3, 0)  # [page, head, tile, key, group, (scale, minimum)]
    k[...] = 0
    k[0, 0, 0, 0, :, 1] = 21 * np.log(2) / D
    v[..., 0] = g.uniform(*scales, v.shape[:-1])
    if odd_key is not None:
        at = (odd_key // page, 0, odd_key % page // 16, odd_key % 16)
        v[at][0, 0] = odd_scale
        if odd_scale > 100:
            k[at][:, 1] = -60 / D
    v[..., 1] = -7.5 * v[..., 0]
    pool[..., 16 * D:] = pairs.reshape(num, 1, page // 16, -1).view(np.uint8)
    table = np.arange(num, dtype=np.int32)[None]
    q = torch.ones(1, Hq, 1, D, dtype=torch.bfloat16)
    for out_dtype in types:
        O, lse, bO, bL = decode_bound(q, pool, table, [n], 1.0, out_dtype == torch.float32)
        out, ls = run_decode(q[:, :, 0].contiguous(), pool, table, [n], 1.0, chunk=1 << 20, out_dtype=out_dtype)
        assert_within(out[:, :, None], O, bO, f"O {out_dtype}")
        assert_within(ls[:, :, None], lse, bL, f"lse {out_dtype}")


@pytest.mark.parametrize("D,Hq", [(64, 1), (64, 8), (128, 1), (128, 8), (128, 16)])
def test_decode_q4_long_slices_in_fp32(D, Hq):
    """131072 keys added to one accumulator: terms 2^-23 of the first one's size each, thousands of sums."""
    check_first_key_leads(131072, D, Hq, (0.2, 0.6), [torch.float32])


@pytest.mark.parametrize("n,odd_key,odd_scale,scales", [
    (131072, 0, 2.5, (0.2, 0.6)),        # one scale a few times the others'
    (16384, 8000, 2.5, (0.2, 0.6)),
    (16384, None, None, (1.5, 2.5)),     # scales on both sides of a power of two
    (131072, 500, 8000.0, (2e-4, 4e-4)),   # a scale far above all others, of a key that hardly counts
    (16384, 9001, 8000.0, (2e-4, 4e-4)),
])
@pytest.mark.parametrize("D,Hq", [(64, 1), (128, 8)])
def test_decode_q4_scales_of_v_that_differ(n, odd_key, odd_scale, scales, D, Hq):
    check_first_key_leads(n, D, Hq, scales, [torch.bfloat16, torch.float32], odd_key, odd_scale)


@pytest.mark.parametrize("B,Hq,Hkv", [(40, 16, 4), (400, 4, 2), (1100, 2, 1)])
def test_decode_q4_many_sequences(B, Hq, Hkv):
    g = np.random.default_rng(B)
    lens = [int(x) for x in g.integers(0, 60, B)]
    check_decode(B, Hq, Hkv, 1, 64, 16, lens, seed=B, poison_rest=False)


def test_decode_q4_long_matches_the_reference():
    check_decode(2, 4, 1, 1, 128, 64, [40000, 12345], seed=3, poison_rest=False)


def test_decode_q4_is_reproducible_and_agrees_across_lq():
    pool = make_pool(400, 2, 16, 128, 4)
    table, _ = make_table([3000, 1500], 16, 400, 5)
    q = torch.randn(2, 8, 1, 128).to(torch.bfloat16)
    a = run_decode(q[:, :, 0].contiguous(), pool, table, [3000, 1500], 0.09)
    b = run_decode(q[:, :, 0].contiguous(), pool, table, [3000, 1500], 0.09)
    c = run_decode(q, pool, table, [3000, 1500], 0.09)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(a[0], c[0][:, :, 0]) and torch.equal(a[1], c[1][:, :, 0])


@pytest.mark.parametrize("Lq,n", [(1, 20), (1, 3000), (2, 40), (4, 3000)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_decode_q4_nan_queries_stay_in_their_rows(Lq, n, bad):
    pool, (table, _) = make_pool(200, 2, 16, 64, 4), make_table([n], 16, 200, 4)
    q = torch.randn(1, 8, Lq, 64, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16)
    hurt = q.clone()
    hurt[0, 3, 0, 5] = bad
    O, lse = run_decode(q, pool, table, [n], 0.125)
    o, ls = run_decode(hurt, pool, table, [n], 0.125)
    assert o[0, 3, 0].isnan().all() and ls[0, 3, 0].isnan()
    o[0, 3, 0], ls[0, 3, 0] = O[0, 3, 0], lse[0, 3, 0]
    assert torch.equal(o, O) and torch.equal(ls, lse)


def test_decode_q4_bad_lengths_and_pages_are_flagged():
    pool = dev(make_pool(4, 2, 16, 64, 4))
    q = dev(torch.randn(2, 4, 64).to(torch.bfloat16))
    table = dev(np.array([[0, 1], [2, 3]], np.int32))
    for t, lens in ((table, [33, 5]), (table, [-1, 5]), (dev(np.array([[0, 4], [2, 3]], np.int32)), [20, 5]),
                    (dev(np.array([[-1, 1], [2, 3]], np.int32)), [20, 5])):
        AB.attn_decode_q4(q, pool, t, i32(lens))
        assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_BOUNDS
    AB.attn_decode_q4(q, pool, dev(np.array([[0, -1], [2, 99]], np.int32)), i32([16, 16]))  # entries no key needs
    assert AB.attn_get_device_status() == AB.ATTN_OK


def test_decode_q4_timeout_is_reported_and_the_next_call_is_right(monkeypatch):
    pool = make_pool(2000, 2, 16, 128, 4)
    table, _ = make_table([16000, 15000], 16, 2000, 5)
    q = torch.randn(2, 8, 128).to(torch.bfloat16)
    a = run_decode(q, pool, table, [16000, 15000], 0.09, chunk=1 << 14)
    monkeypatch.setenv("ATTN_FAULT_INJECT", "skip_arrive")
    AB.attn_decode_q4(dev(q), dev(pool), dev(table), i32([16000, 15000]), scale=0.09, chunk=1 << 14)
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("ATTN_FAULT_INJECT")
    b = run_decode(q, pool, table, [16000, 15000], 0.09, chunk=1 << 14)
    assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("first", [AB.ATTN_ERR_DEVICE_POOL, AB.ATTN_ERR_DEVICE_BOUNDS])
def test_a_timeout_is_told_whatever_was_recorded_before(monkeypatch, first):
    # An unread status of another kind, a decode that gives up over rows split between CTAs, and one that follows.
    pool, (table, _) = make_pool(1000, 1, 16, 128, 4), make_table([16000], 16, 1000, 5)
    args = (torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16), pool, table, [16000], 0.09)
    a = run_decode(*args, chunk=1 << 12)
    d_args = dev(args[0]), dev(pool), dev(table), i32([16000])
    new = i32([1 if first == AB.ATTN_ERR_DEVICE_POOL else -1])
    AB.attn_page_step(i32([0]), i32([-1])[None], i32([0]), i32([0]), 16, new_lens=new)
    monkeypatch.setenv("ATTN_FAULT_INJECT", "skip_arrive")
    AB.attn_decode_q4(*d_args, scale=0.09, chunk=1 << 12)
    monkeypatch.delenv("ATTN_FAULT_INJECT")
    AB.attn_page_step(i32([0]), i32([-1])[None], i32([0]), i32([0]), 16, new_lens=new)
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_TIMEOUT
    for _ in range(2):
        b = run_decode(*args, chunk=1 << 12)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("Hq,Hkv,Lq,D", [(8, 2, 1, 128), (8, 2, 1, 64), (16, 2, 1, 128), (32, 2, 2, 64), (24, 2, 3, 128)])
def test_decode_q4_leaves_its_workspace_zero(Hq, Hkv, Lq, D):
    """Rows in one CTA, in a few and in all of them, sequences without keys: whatever counts and partials a call writes it
    takes back, and the next call starts from there."""
    ws = AB.attn_decode_q4_workspace(Hq, Hkv, D, Lq=Lq, device=DEV)
    pool, q = dev(make_pool(700, Hkv, 16, D, 4)), dev(torch.randn(3, Hq, Lq, D).to(torch.bfloat16))
    for lens in ([1, 0, 16], [700, 64, 0], [5000, 3000, 1000], [9, 9000, 1]):
        table = dev(make_table(lens, 16, 700, 5)[0])
        for chunk in (0, 1, 600):
            for dtype in (torch.bfloat16, torch.float32):
                AB.attn_decode_q4(q, pool, table, i32(lens), chunk=chunk, out_dtype=dtype, workspace=ws)
                assert AB.attn_get_device_status() == AB.ATTN_OK and (ws == 0).all(), (lens, chunk, dtype)


def test_cache_calls_refuse_what_they_would_misread():
    pool = dev(make_pool(4, 2, 16, 64, 4))
    q, table, lens = dev(torch.randn(1, 4, 64).to(torch.bfloat16)), i32([0, 1])[None], i32([20])
    k = dev(torch.randn(3, 2, 64).to(torch.bfloat16))
    for args in ((k, k, pool, i32([0, 1])), (k, k[:2], pool, i32([0, 1, 2])), (k[:, :1], k[:, :1], pool, i32([0, 1, 2])),
                 (k, k, pool[..., :1000], i32([0, 1, 2])), (k, k.transpose(1, 2), pool, i32([0, 1, 2])),
                 (k, k, pool, i32([0, 1, 2]).long()), (k.float(), k, pool, i32([0, 1, 2]))):
        with pytest.raises((ValueError, TypeError)):
            AB.attn_kv_append_q4(*args)
    for kw in (dict(cu_k=i32([0, 3, 4])), dict(kv_starts=i32([0, 0])), dict(total_k=4, k_out=k), dict(block_table=table[0])):
        with pytest.raises((ValueError, TypeError)):
            AB.attn_kv_gather_q4(**{**dict(pool=pool, block_table=table, cu_k=i32([0, 3]), total_k=3), **kw})
    for kw in (dict(q=q.float()), dict(q=q.cpu()), dict(kv_lens=lens.long()), dict(kv_lens=i32([1, 2])),
               dict(block_table=table[0]), dict(out=torch.empty(1, 4, 128, dtype=torch.bfloat16, device=DEV)),
               dict(lse=torch.empty(4, device=DEV)), dict(out_dtype=torch.float16), dict(pool=pool.view(4, 2, -1)),
               dict(workspace=torch.zeros(8, device=DEV))):
        with pytest.raises((ValueError, TypeError)):
            AB.attn_decode_q4(**{**dict(q=q, pool=pool, block_table=table, kv_lens=lens), **kw})
    with pytest.raises(AB.AttnError) as e:
        AB.attn_decode_q4(q[:, :3].contiguous(), pool, table, lens)  # 3 query heads over 2
    assert e.value.status == AB.ATTN_ERR_INVALID_ARG
    assert AB.attn_get_device_status() == AB.ATTN_OK


def test_decode_q4_workspace_is_zeroed_on_the_calls_stream():
    # the library's workspace is made by a call on a side stream, while the default stream is busy
    pool, q = dev(make_pool(64, 1, 16, 64, 7)), dev(torch.randn(1, 4, 64).to(torch.bfloat16))
    args = (q, pool, i32(range(64))[None], i32([1024]))
    want = AB.attn_decode_q4(*args, workspace=AB.attn_decode_q4_workspace(4, 1, 64))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    AB.attn_release_workspace()
    torch.cuda._sleep(100_000_000)
    with torch.cuda.stream(side):
        for _ in range(3):
            got = AB.attn_decode_q4(*args)
            side.synchronize()
            assert torch.equal(want[0].cpu(), got[0].cpu()) and torch.equal(want[1].cpu(), got[1].cpu())
    torch.cuda.synchronize()
    assert AB.attn_get_device_status() == AB.ATTN_OK


def test_decode_q4_does_not_make_its_workspace_inside_a_capture():
    pool, q = dev(make_pool(1, 1, 16, 64, 4)), dev(torch.randn(1, 1, 64).to(torch.bfloat16))
    args = (q, pool, i32([0])[None], i32([5]))
    want = AB.attn_decode_q4(*args)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    AB.attn_release_workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(AB.AttnError) as e:
            AB.attn_decode_q4(*args, out=out, lse=lse)
        out.fill_(3)
    assert e.value.status == AB.ATTN_ERR_INVALID_ARG
    graph.replay()  # the capture itself was left intact
    torch.cuda.synchronize()
    assert (out == 3).all()
    assert torch.equal(AB.attn_decode_q4(*args)[0], want[0])


def test_decode_q4_workspace_too_small_is_refused():
    pool, q = dev(make_pool(1, 1, 16, 64, 4)), dev(torch.randn(1, 1, 64).to(torch.bfloat16))
    ws = torch.zeros(1024, dtype=torch.uint8, device=DEV)
    with pytest.raises(AB.AttnError) as e:
        AB.attn_decode_q4(q, pool, i32([0])[None], i32([3]), workspace=ws)
    assert e.value.status == AB.ATTN_ERR_SCRATCH_TOO_SMALL


# ---------------------------------------------------------------- together

class Engine:
    """A small serving engine's state: pages, pool, and the tensors of a step of up to `room` tokens."""

    def __init__(self, B, Hq, Hkv, D, page, num_pages, width, room):
        self.Hq, self.Hkv, self.D, self.page, self.B, self.room = Hq, Hkv, D, page, B, room
        self.lens, self.table = i32([0] * B), torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        self.free, self.count = i32(range(num_pages)), i32([num_pages])
        self.pool = AB.attn_kv_q4_pool(num_pages, Hkv, page, D, DEV)
        self.new, self.slots, self.pos = i32([0] * B), i32([0] * room), i32([0] * room)
        self.cu = i32([0] * (B + 1))
        self.rope = tuple(x.to(DEV) for x in rope_tables(width * page, D)) + ("half",)
        self.w = (1 + 0.1 * torch.randn(2, D, device=DEV)).to(torch.bfloat16)
        self.qkv = torch.zeros(room, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
        self.q, self.k = (torch.empty(room, h, D, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv))
        self.ws = AB.attn_decode_q4_workspace(Hq, Hkv, D, device=DEV)
        self.out = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.zeros(B, Hq, device=DEV)

    def prefix(self):
        AB.attn_page_step(self.lens, self.table, self.free, self.count, self.page, new_lens=self.new,
                          slots=self.slots, positions=self.pos, cu_new=self.cu)
        AB.attn_qk_norm_rope(self.qkv[:, :self.Hq], self.qkv[:, self.Hq:self.Hq + self.Hkv], self.w[0], self.w[1],
                             self.rope, self.pos, q_out=self.q, k_out=self.k)
        AB.attn_kv_append_q4(self.k, self.qkv[:, self.Hq + self.Hkv:], self.pool, self.slots)

    def decode(self):
        self.prefix()
        AB.attn_decode_q4(self.q[:self.B], self.pool, self.table, self.lens, out=self.out, lse=self.lse,
                          workspace=self.ws)

    def check(self, q):
        """The decode's output against fp64 over the values now in the cache."""
        O, lse, bO, bL = decode_bound(q[:, :, None].cpu(), self.pool.cpu().numpy(), self.table.cpu().numpy(),
                                      self.lens.tolist(), self.D ** -0.5, False)
        assert_within(self.out[:, :, None], O, bO)
        assert_within(self.lse[:, :, None], lse, bL)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64)])
def test_a_serving_run(Hq, Hkv, D):
    """Prompts through prefill over the cache, decode steps through a captured graph, drafts taken back, a request that
    ends and one that takes its place; each step against fp64 over the values in the cache, and those against the rows."""
    torch.manual_seed(1)
    B, room = 3, 96
    e = Engine(B, Hq, Hkv, D, 16, 40, 12, room)
    # prompts of 30, 0 and 41 tokens (25 rows of padding)
    e.new.copy_(i32([30, 0, 41]))
    e.qkv.normal_()
    e.prefix()
    assert e.lens.tolist() == [30, 0, 41] and e.cu.tolist() == [0, 30, 30, 71]
    kd, vd = AB.attn_kv_gather_q4(e.pool, e.table, e.cu, 71)
    u, s, m = oracle.quantise_q4(e.k[:71])
    assert torch.equal(kd.cpu(), torch.from_numpy(oracle.values_q4(u, s, m)).float().to(torch.bfloat16))
    out, _ = AB.attn_fwd_varlen(e.q[:71], kd, vd, e.cu, e.cu, 41, 41)
    O, _ = oracle.attention_varlen(e.q[:71].cpu(), kd.cpu(), vd.cpu(), e.cu.cpu().numpy(), e.cu.cpu().numpy(),
                                   D ** -0.5, True)
    assert np.abs(out.double().cpu().numpy() - O).max() < 2e-2  # the prefill kernel's own bar
    # decode: one token each, the middle request gets its first
    e.new.copy_(i32([1, 1, 1]))
    s0 = torch.cuda.Stream()
    s0.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s0):
        e.decode()
    for step in range(20):
        e.qkv.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert e.lens.tolist() == [31 + step, 1 + step, 42 + step]
        assert e.pos.tolist()[:4] == [30 + step, step, 41 + step, -1]
        e.check(e.q[:B])
    # take four tokens of request 0 back, end request 1, start another in its place with 9 tokens
    e.new.copy_(i32([0, 9, 0]))
    AB.attn_page_step(e.lens, e.table, e.free, e.count, e.page, new_lens=e.new, keep_lens=i32([46, 0, 61]),
                      slots=e.slots, positions=e.pos, cu_new=e.cu)
    assert e.lens.tolist() == [46, 9, 61] and e.count.item() == 40 - 3 - 1 - 4
    e.new.copy_(i32([1, 1, 1]))
    graph.replay()
    torch.cuda.synchronize()
    e.check(e.q[:B])
    assert AB.attn_get_device_status() == AB.ATTN_OK


def test_two_captured_steps_replayed_at_once():
    torch.manual_seed(2)
    engines, graphs = [], []
    for i in range(2):
        e = Engine(2, 8, 2, 128, 16, 700, 300, 2)
        e.pool.copy_(dev(make_pool(700, 2, 16, 128, i)))
        e.new.copy_(i32([3000, 2500]))
        AB.attn_page_step(e.lens, e.table, e.free, e.count, 16, new_lens=e.new)
        e.new.copy_(i32([1, 1]))
        e.qkv.normal_()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            e.decode()
        engines.append((e, st))
        graphs.append(g)
    for _ in range(30):
        for (e, st), g in zip(engines, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for e, _ in engines:
        assert e.lens.tolist() == [3030, 2530]
        e.check(e.q[:2])
    assert AB.attn_get_device_status() == AB.ATTN_OK


@pytest.mark.parametrize("Hq,Hkv,D,Lq,style", [(8, 2, 128, 4, "half"), (4, 4, 64, 3, "interleaved"), (16, 2, 128, 5, "half")])
def test_draft_steps_in_a_graph(Hq, Hkv, D, Lq, style):
    """Steps of Lq draft tokens a request, some of them refused: pages, norm into the decode's layout, rows into the cache,
    decode of all drafts at once, captured as one step; every output against fp64 over the values in the cache."""
    B, page = 3, 16
    g = torch.Generator(device=DEV).manual_seed(Lq)
    lens, keep, new = i32([0] * B), i32([0] * B), i32([Lq] * B)
    table, free, count = torch.full((B, 9), -1, dtype=torch.int32, device=DEV), i32(range(30)), i32([30])
    slots, pos = i32([0] * (B * Lq)), i32([0] * (B * Lq))
    pool = AB.attn_kv_q4_pool(30, Hkv, page, D, DEV)
    rope = tuple(x.to(DEV) for x in rope_tables(9 * page, D)) + (style,)
    w = (1 + 0.1 * torch.randn(2, D, generator=g, device=DEV)).to(torch.bfloat16)
    qkv = torch.zeros(B, Lq, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    q, k = torch.empty(B, Hq, Lq, D, dtype=torch.bfloat16, device=DEV), torch.empty(B, Lq, Hkv, D, dtype=torch.bfloat16, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(B, Hq, Lq, device=DEV)
    ws = AB.attn_decode_q4_workspace(Hq, Hkv, D, Lq=Lq, device=DEV)

    def step():
        x = qkv.transpose(1, 2)  # [B, heads, Lq, D]
        AB.attn_page_step(lens, table, free, count, page, new_lens=new, keep_lens=keep, slots=slots, positions=pos)
        AB.attn_qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], w[0], w[1], rope, pos.view(B, Lq), q_out=q, k_out=k.transpose(1, 2))
        AB.attn_kv_append_q4(k.flatten(0, 1), qkv[:, :, Hq + Hkv:].flatten(0, 1), pool, slots)
        AB.attn_decode_q4(q, pool, table, lens, out=out, lse=lse, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = [0] * B
    for i in range(12):
        taken = [h if i == 0 else h - Lq + (i * (b + 1)) % (Lq + 1) for b, h in enumerate(held)]  # 0 to Lq drafts kept
        keep.copy_(i32(taken))
        qkv.normal_(generator=g)
        graph.replay()
        held = [n + Lq for n in taken]
        assert AB.attn_get_device_status() == AB.ATTN_OK and lens.tolist() == held
        assert pos.view(B, Lq).tolist() == [list(range(n, n + Lq)) for n in taken]
        flat = qkv[:, :, :Hq].reshape(B * Lq, Hq, D)
        ref, bound = norm_ref(oracle.to_f64(flat.cpu()), w[0].cpu(), pos.cpu().numpy(), rope, 1e-6, np.ones(B * Lq, bool))
        assert_within(q.transpose(1, 2).reshape(B * Lq, Hq, D), ref, bound)
        cached, _ = AB.attn_kv_gather_q4(pool, table, i32(range(0, B * Lq + 1, Lq)), B * Lq, kv_starts=i32(taken))
        u, s, m = oracle.quantise_q4(k.flatten(0, 1).cpu())
        assert torch.equal(cached.cpu(), torch.from_numpy(oracle.values_q4(u, s, m)).float().to(torch.bfloat16))
        O, L, bO, bL = decode_bound(q.cpu(), pool.cpu().numpy(), table.cpu().numpy(), held, D ** -0.5, False)
        assert_within(out, O, bO)
        assert_within(lse, L, bL)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (4, 4, 64)])
def test_prefill_of_chunks_over_a_cached_prefix(Hq, Hkv, D):
    """Prompts in chunks: each chunk's rows go into the cache, all keys so far are read back, and the packed prefill runs the
    chunk's queries over them (more keys than queries, a request without new tokens among them)."""
    e = Engine(4, Hq, Hkv, D, 16, 80, 30, 600)
    held = [0] * 4
    for new in ([130, 0, 65, 16], [200, 33, 0, 1], [7, 200, 64, 100]):
        e.new.copy_(i32(new))
        e.qkv.normal_()
        e.prefix()
        held = [a + b for a, b in zip(held, new)]
        cu_q, cu_k = e.cu, i32(np.concatenate([[0], np.cumsum(held)]))
        k, v = AB.attn_kv_gather_q4(e.pool, e.table, cu_k, sum(held))
        n = sum(new)
        out, lse = AB.attn_fwd_varlen(e.q[:n], k, v, cu_q, cu_k, max(new), max(held))
        assert AB.attn_get_device_status() == AB.ATTN_OK
        for b in range(4):
            if new[b] == 0:
                continue
            rows, keys = slice(int(cu_q[b]), int(cu_q[b + 1])), slice(sum(held[:b]), sum(held[:b + 1]))
            kk, vv, _, _ = oracle.read_q4(e.pool.cpu().numpy(), e.table[b].cpu().numpy(), 0, held[b])
            for x, got in ((kk, k[keys]), (vv, v[keys])):  # what the cache holds, rounded once
                assert torch.equal(got.cpu(), torch.from_numpy(x).float().to(torch.bfloat16))
            for h in range(Hq):
                o, _ = oracle.attention_head(oracle.to_f64(e.q[rows, h].cpu()), oracle.to_f64(k[keys, h // (Hq // Hkv)].cpu()),
                                             oracle.to_f64(v[keys, h // (Hq // Hkv)].cpu()), D ** -0.5, causal=True)
                assert np.abs(out[rows, h].double().cpu().numpy() - o).max() < 2e-2  # the prefill kernel's own bar


@pytest.mark.parametrize("D", [64, 128])
def test_pool_offsets_past_32_bits(D):
    """The last pages of a pool of over 4 GiB: written, read back and attended to like the first ones of a small one."""
    Hkv, page, n = 4, 64, 300
    page_bytes = AB.attn_kv_q4_page_bytes(page, Hkv, D)
    num_pages = (5 << 30) // page_bytes
    need = -(-n // page)
    assert (num_pages - need) * page_bytes > 1 << 32
    g = torch.Generator().manual_seed(D)
    k, v = dev(torch.randn(2, n, Hkv, D, generator=g).to(torch.bfloat16))
    q = dev(torch.randn(1, 8, D, generator=g).to(torch.bfloat16))
    got = []
    for pages in (need, num_pages):
        pool = AB.attn_kv_q4_pool(pages, Hkv, page, D, DEV)
        table = torch.arange(pages - need, pages, dtype=torch.int32, device=DEV)[None]
        pos = torch.arange(n, device=DEV)
        slots = table[0, pos // page] * page + (pos % page).to(torch.int32)
        AB.attn_kv_append_q4(k, v, pool, slots)
        got.append((*AB.attn_kv_gather_q4(pool, table, i32([0, n]), n), *AB.attn_decode_q4(q, pool, table, i32([n]))))
        assert AB.attn_get_device_status() == AB.ATTN_OK
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_norm_without_rotation_or_positions():
    q = dev(torch.randn(5, 3, 64).to(torch.bfloat16))
    qo, ko = AB.attn_qk_norm_rope(q, None)
    assert ko is None
    ref, bound = norm_ref(oracle.to_f64(q), None, np.zeros(5, int), None, 1e-6, np.ones(5, bool))
    assert_within(qo, ref, bound)


def test_decode_q4_rows_of_every_width_over_a_long_capacity():
    """16 query rows a CTA: taken from the block table's capacity, whatever the lengths."""
    lens, page = [70, 0, 33], 16
    pool = make_pool(10, 2, page, 64, 8)
    table, _ = make_table(lens, page, 10, 8, width=120000)
    for Hq, Lq in ((24, 1), (8, 5), (2, 16)):
        q = torch.randn(3, Hq, Lq, 64, generator=torch.Generator().manual_seed(Hq)).to(torch.bfloat16)
        for f32 in (False, True):
            O, lse, bO, bL = decode_bound(q, pool, table, lens, 0.125, f32)
            out, ls = run_decode(q, pool, table, lens, 0.125, out_dtype=torch.float32 if f32 else torch.bfloat16)
            assert_within(out, O, bO)
            assert_within(ls, lse, bL)


@pytest.mark.parametrize("Hq,Lq", [(24, 1), (18, 1), (8, 5), (2, 16), (6, 13)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_q4_wide_rows_split_between_many_ctas(D, Hq, Lq):
    """16 query rows a CTA over a long capacity, a sequence of thousands of keys split into pieces that are merged four at a
    time and singly, beside short and empty ones; by the default split too."""
    lens, page = [6000, 0, 33, 1, 700], 16
    pool = make_pool(430, 2, page, D, 8)
    table, _ = make_table(lens, page, 430, 8, width=120000)
    q = torch.randn(5, Hq, Lq, D, generator=torch.Generator().manual_seed(Hq)).to(torch.bfloat16)
    for dtype in (torch.bfloat16, torch.float32):
        O, lse, bO, bL = decode_bound(q, pool, table, lens, 0.1, dtype == torch.float32)
        seen = []
        for chunk in (0, 256, 1000, 1 << 20):
            out, ls = run_decode(q, pool, table, lens, 0.1, chunk=chunk, out_dtype=dtype)
            assert_within(out, O, bO, f"O {dtype} {chunk}")
            assert_within(ls, lse, bL, f"lse {dtype} {chunk}")
            again = run_decode(q, pool, table, lens, 0.1, chunk=chunk, out_dtype=dtype)
            assert torch.equal(out, again[0]) and torch.equal(ls, again[1])
            seen.append(out)
        assert not torch.equal(seen[1], seen[3])  # split indeed


def test_side_stream_gives_the_same_bits():
    torch.manual_seed(3)
    pool = dev(make_pool(100, 2, 16, 64, 1))
    table = dev(make_table([700, 500], 16, 100, 2)[0])
    q, lens = dev(torch.randn(2, 8, 64).to(torch.bfloat16)), i32([700, 500])
    a = AB.attn_decode_q4(q, pool, table, lens)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    b = AB.attn_decode_q4(q, pool, table, lens, stream=st)
    st.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decodes_of_several_streams_at_once():
    """Four streams' decodes of different shapes, each with a workspace of its own, beside a prefill that holds SMs: whichever
    CTAs start first, the bits are those of the calls one after another."""
    cases = []
    for i, (B, Hq, Hkv, Lq, D, hi) in enumerate([(1, 32, 8, 1, 128, 9000), (6, 16, 16, 1, 64, 1500), (3, 8, 2, 4, 128, 4000),
                                                  (40, 8, 2, 1, 64, 300)]):
        g = np.random.default_rng(i)
        lens = [int(x) for x in g.integers(0, hi + 1, B - 1)] + [hi]
        num = sum(-(-n // 16) for n in lens)
        pool, table = dev(make_pool(num, Hkv, 16, D, i)), dev(make_table(lens, 16, num, i)[0])
        q = dev(torch.randn(B, Hq, Lq, D, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16))
        cases.append((q, pool, table, i32(lens), AB.attn_decode_q4_workspace(Hq, Hkv, D, Lq=Lq, device=DEV), torch.cuda.Stream()))
    want = [AB.attn_decode_q4(*c[:4], workspace=c[4]) for c in cases]
    x = dev(torch.randn(3, 2, 8, 2048, 128).to(torch.bfloat16))
    side = torch.cuda.Stream()
    outs = [[(torch.empty_like(w[0]), torch.empty_like(w[1])) for _ in range(25)] for w in want]
    torch.cuda.synchronize()
    for n in range(25):
        AB.attn_fwd(x[0], x[1], x[2], stream=side)
        for c, w in zip(cases, outs):
            AB.attn_decode_q4(*c[:4], out=w[n][0], lse=w[n][1], workspace=c[4], stream=c[5])
    torch.cuda.synchronize()
    assert AB.attn_get_device_status() == AB.ATTN_OK
    for w, got in zip(want, outs):
        assert all(torch.equal(o, w[0]) and torch.equal(ls, w[1]) for o, ls in got)


FIRST_CALLS = """
import torch
from attention_attn_fwd_06_gb300 import binding as AB
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
lens, table, free, count, new = i32([0] * 3), i32([[-1, -1]] * 3), i32(range(8)), i32([8]), i32([5, 17, 0])
slots, pos, cu = i32([0] * 22), i32([0] * 22), i32([0] * 4)
x = torch.randn(22, 2, 64, device="cuda").to(torch.bfloat16)
pool = torch.zeros(8, 2, 1, 18 * 64, dtype=torch.uint8, device="cuda")
cos = torch.randn(32, 32, device="cuda")
q, k, v, out, lse = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(x[:3]), torch.empty(3, 2, device="cuda")
ws = AB.attn_decode_q4_workspace(2, 2, 64)  # (a size only: nothing has run)

def step():
    AB.attn_page_step(lens, table, free, count, 16, new_lens=new, slots=slots, positions=pos, cu_new=cu)
    AB.attn_qk_norm_rope(x, None, rope=(cos, cos, "half"), positions=pos, q_out=q)
    AB.attn_kv_append_q4(q, x, pool, slots)
    AB.attn_kv_gather_q4(pool, table, cu, 22, k_out=k, v_out=v)
    AB.attn_decode_q4(q[:3], pool, table, lens, out=out, lse=lse, workspace=ws)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
got = [t.clone() for t in (lens, table, slots, pos, cu, q, k, v, out, lse)]
lens.zero_(), table.fill_(-1), free.copy_(i32(range(8))), count.fill_(8), pool.zero_()
step()
assert AB.attn_get_device_status() == AB.ATTN_OK
assert all(torch.equal(a, b) for a, b in zip(got, (lens, table, slots, pos, cu, q, k, v, out, lse)))
assert lens.tolist() == [5, 17, 0] and lse[2].isneginf().all()
"""


def test_first_calls_of_a_process_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=120,
                       cwd=pathlib.Path(__file__).parents[1])
    assert r.returncode == 0, r.stderr
