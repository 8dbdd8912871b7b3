"""GPU parity of a draft step's calls at the edges of what they allow: rows of probabilities that end inside a 16-byte load or are
very long, queries and values that are not numbers, rotary tables of large bases."""
import math
import pathlib
import subprocess
import sys
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import oracle
from attention_attn_fwd_06_gb300 import binding as AB
from attention_attn_fwd_06_gb300.build import build
from tests.test_gpu_drafts import Cache, bf16, i32, probabilities

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build()
    AB.load()
    AB.attn_get_device_status()


# ---------------------------------------------------------------- verification of drafts

def padded(x, fill):
    """x [..., V] as a view of rows on 16 bytes, padded past V with `fill`."""
    V = x.shape[-1]
    wide = torch.full((*x.shape[:-1], (V + 8) // 8 * 8), fill, dtype=x.dtype, device=DEV)
    wide[..., :V] = x.to(DEV)
    assert wide.data_ptr() % 16 == 0
    return wide[..., :V]


LAST_NUMBERS = [0.0, 0.3, 1 - 2.0 ** -24, 1.0, float("inf"), float("nan")]


@pytest.mark.parametrize("form", ["drawn", "point", "all", "packed"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 33, 37, 260, 1003, 50257])
def test_verify_drafts_rows_that_end_inside_a_load(V, dtype, form):
    """Padding past the last token would win every draw; the last tokens hold weight; numbers up to 1 and past it."""
    g = np.random.default_rng(V)
    B = len(LAST_NUMBERS)
    q = torch.from_numpy(probabilities(B, V, g)).view(B, 1, V)
    p = torch.from_numpy(probabilities(2 * B, V, g)).view(B, 2, V)
    q[..., -5:], p[..., -5:] = 0.25 * p[:, :1, -5:] + 0.001, p[..., -5:] + 0.002
    p, q = p.to(dtype), q.to(dtype)
    draft = (q - p[:, :1]).float().argmax(-1)  # where the draft's row is furthest above the target's
    u = np.full((B, 2), 1 - 2.0 ** -24, np.float32)
    if form == "all":
        u[:, 0] = 0.0
    u[:, 1] = LAST_NUMBERS
    rows, kw = padded(p, 60000.0), {}
    if form == "packed":
        rows, kw["cu_target"] = rows.flatten(0, 1), i32(2 * np.arange(B + 1))
        assert rows.stride(0) % 8 == 0
    if form != "point":
        kw["draft_probs"] = padded(q, -60000.0)
    tokens, accepted, _ = AB.attn_verify_drafts(i32(draft), rows, torch.from_numpy(u).to(DEV), **kw)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    for b in range(B):
        stand, token = oracle.verify_drafts(draft[b].tolist(), p[b].float().numpy(), u[b].tolist(),
                                            None if form == "point" else q[b].float().numpy())
        assert accepted[b] == stand and tokens[b].tolist() == draft[b, :stand].tolist() + [token] + [-1] * (1 - stand), LAST_NUMBERS[b]
    if form == "all":
        assert (accepted == 1).all()


@pytest.mark.parametrize("last", [1.0, 2.0, float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 300, 1003, 70000, 600000])
def test_verify_drafts_numbers_of_one_and_more_draw_the_last_token_with_any_weight(V, dtype, last):
    """The last weights are far below the sum's last bit, whatever the order that the others are added up in."""
    g = torch.Generator(device=DEV).manual_seed(V)
    B = 40 if V < 100000 else 6
    p = torch.rand(B, 1, V, generator=g, device=DEV).to(dtype)
    p[..., -4:] = 0
    p[..., -3] = 1e-30
    u = torch.full((B, 1), last, device=DEV)
    for padding in (0, 3):
        wide = torch.full((B, 1, V + padding), 1.0, dtype=dtype, device=DEV)
        wide[..., :V] = p
        tokens, _, _ = AB.attn_verify_drafts(torch.zeros(B, 0, dtype=torch.int32, device=DEV), wide[..., :V], u)
        assert tokens.flatten().tolist() == [V - 3] * B and AB.attn_get_device_status() == AB.ATTN_OK


@pytest.mark.parametrize("V", [4, 5000])
def test_verify_drafts_weights_of_the_smallest_numbers(V):
    """Multiples of fp32's smallest number, and numbers whose share of their sum is one: exact."""
    w = np.zeros(V, np.float32)
    w[[0, 1, V - 2, V - 1]] = np.array([3, 5, 7, 1]) * 2.0 ** -149
    p = torch.from_numpy(w).view(1, 1, V).to(DEV)
    for u, want in ((0.0, 0), (0.125, 0), (0.25, 1), (0.5, V - 2), (0.9375, V - 1), (1.0, V - 1)):
        tokens, _, _ = AB.attn_verify_drafts(torch.zeros(1, 0, dtype=torch.int32, device=DEV), p, torch.tensor([[u]], device=DEV))
        assert tokens.item() == want and AB.attn_get_device_status() == AB.ATTN_OK


@pytest.mark.parametrize("odd", [None, float("inf")], ids=["finite", "with an infinity"])
def test_verify_drafts_sums_of_half_a_billion_equal_weights(odd):
    """0.1 for the first half of the row and 1/16, whose sums are exact, for the rest.  A sum that is off by d of the first half's
    moves a token of the second half by d V 0.8 (1 - u): within 2^-34 of it not by one, as the tokens' shares of u are 0.3 to 0.7."""
    V, half = (1 << 29) + 77, 1 << 28
    p = torch.full((1, 1, V), 0.1, device=DEV)
    p[..., half:] = 0.0625
    first = half
    if odd is not None:
        p[..., 5] = odd  # counts as nothing, and every weight is looked at
        first -= 1
    w, scale = float(np.float32(0.1)).as_integer_ratio()
    x = scale // 16
    total = first * w + (V - half) * x  # of 1 / scale
    found = 0
    for k in range(1, 40):
        u = float(np.float32(0.62 + 0.0093 * k))
        num, den = u.as_integer_ratio()
        want, part = divmod(num * total - den * first * w, den * x)
        if not 0.3 < part / (den * x) < 0.7:
            continue
        found += 1
        tokens, _, _ = AB.attn_verify_drafts(torch.zeros(1, 0, dtype=torch.int32, device=DEV), p, torch.tensor([[u]], device=DEV))
        assert tokens.item() == half + want
    assert found > 8 and AB.attn_get_device_status() == AB.ATTN_OK


# ---------------------------------------------------------------- decode over pages

def decode(c, q, new, f32=False, gap=0):
    cu = i32(gap + np.concatenate([[0], np.cumsum(new)]))
    o, ls = AB.attn_decode_multi_paged(q.to(DEV), *c.on_gpu(), cu, max(new), out_dtype=torch.float32 if f32 else torch.bfloat16)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    return o, ls


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens", [[20], [9000, 300]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,new", [(8, 1), (11, 3), (8, 8), (13, 5), (16, 8)])  # 8, 33, 64, 65 and 128 rows of a kv head
def test_decode_multi_paged_nan_queries_stay_in_their_rows(Hq, new, D, lens, bad):
    c = Cache(lens, 1, D, 16, 3)
    news = [new] + [1] * (len(lens) - 1)
    q = bf16((sum(news), Hq, D), Hq)
    hurt = q.clone()
    hurt[0, 3, 5] = bad
    for f32 in (False, True):
        O, lse = decode(c, q, news, f32)
        o, ls = decode(c, hurt, news, f32)
        assert o[0, 3].isnan().all() and ls[0, 3].isnan()
        o[0, 3], ls[0, 3] = O[0, 3], lse[0, 3]
        assert torch.equal(o, O) and torch.equal(ls, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,new", [(2, 4), (16, 8)])
def test_decode_multi_paged_tokens_without_keys_are_zero_beside_nan_values(Hq, new, D):
    """A sequence of fewer keys than new tokens: the first ones see none, whatever the others' values are."""
    c = Cache([new - 2], 1, D, 16, 3)
    c.v[c.table[0, 0], :, new - 3] = float("nan")
    q = bf16((new, Hq, D), 1)
    for f32 in (False, True):
        o, ls = decode(c, q, [new], f32)
        assert (o[:2] == 0).all() and torch.isneginf(ls[:2]).all() and ls[2:].isfinite().all() and o[new - 1].isnan().all()


@pytest.mark.parametrize("Hq", [8, 64, 128, 136])  # 4, 32, 64 and 68 rows of a kv head
def test_decode_multi_paged_timeout_leaves_every_warp_together(monkeypatch, Hq):
    """D = 64: CTA 0 withholds an arrival, so a bounded wait runs out after a second; all warps wind down, the next call is right."""
    c = Cache([16384, 16000], 8, 64, 64, 3)
    args = bf16((8, Hq, 64), 1).to(DEV), *c.on_gpu(), i32([0, 4, 8]), 4
    want, wl = AB.attn_decode_multi_paged(*args)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    monkeypatch.setenv("ATTN_FAULT_INJECT", "skip_arrive")
    AB.attn_decode_multi_paged(*args)
    assert AB.attn_get_device_status() == AB.ATTN_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("ATTN_FAULT_INJECT")
    out, lse = AB.attn_decode_multi_paged(*args)
    assert AB.attn_get_device_status() == AB.ATTN_OK
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_calls_of_several_host_threads_at_once():
    """In a process of its own, so that the threads' calls are the first ones: each gets its own results."""
    code = """
import threading, torch
from attention_attn_fwd_06_gb300 import binding as AB
AB.load()
D = "cuda:0"
g = torch.Generator().manual_seed(1)
i32 = lambda *s, hi=100: torch.randint(0, hi, s, generator=g, dtype=torch.int32).to(D)
probs = [torch.softmax(torch.randn(8, 5, V, generator=g), -1).to(D) for V in (1000, 1001, 70000, 300000)]
drafts, u = i32(8, 4), torch.rand(8, 5, generator=g).to(D)
q = torch.randn(1, 2, 200, 64, generator=g).bfloat16().to(D)
gate, got, lock = threading.Barrier(12), {}, threading.Lock()
torch.cuda.synchronize()

def page():
    lens, table, free, count = (torch.zeros(4, dtype=torch.int32, device=D), torch.zeros(4, 8, dtype=torch.int32, device=D),
                                torch.arange(32, dtype=torch.int32, device=D), torch.tensor([32], dtype=torch.int32, device=D))
    AB.attn_page_step(lens, table, free, count, 16, new_lens=torch.full((4,), 20, dtype=torch.int32, device=D))
    return lens, table

def work(i):
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        gate.wait()
        outs = []
        for _ in range(20):
            if i < 8:
                outs.append(AB.attn_verify_drafts(drafts, probs[i % 4], u)[:2])
            elif i < 10:
                outs.append(page())
            else:
                outs.append(AB.attn_fwd(q, q, q))
        stream.synchronize()
    with lock:
        got[i] = outs

threads = [threading.Thread(target=work, args=(i,)) for i in range(12)]
[t.start() for t in threads]
[t.join() for t in threads]
assert len(got) == 12 and AB.attn_get_device_status() == AB.ATTN_OK
want = [AB.attn_verify_drafts(drafts, p, u)[:2] for p in probs]
for i, outs in got.items():
    ref = want[i % 4] if i < 8 else page() if i < 10 else AB.attn_fwd(q, q, q)
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, ref)), i
print("alike")
"""
    run = subprocess.run([sys.executable, "-c", code], cwd=pathlib.Path(__file__).parent.parent, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "alike" in run.stdout, run.stderr[-2000:]


# ---------------------------------------------------------------- rotary tables

PI = Decimal("3.141592653589793238462643383279502884197169399375105820974944592307816406286")


def exact_frequencies(R, base, scaling):
    """Radians a position, to some 70 digits."""
    log = Decimal(base).ln()
    if scaling and scaling[0] == "base":
        log += Decimal(R) / (R - 2) * Decimal(scaling[1]).ln()
    return [(-Decimal(2 * i) / R * log).exp() / (Decimal(scaling[1]) if scaling and scaling[0] == "linear" else 1)
            for i in range(R // 2)]


@pytest.mark.parametrize("base,R,scaling", [
    (1e8, 112, None), (1e8, 80, ("linear", 4.0)), (1e4, 96, ("base", 1e10)), (1e20, 128, None),
    (1e20, 112, ("linear", 1e-12)),  # pairs of many turns a position: the angle's own bound counts
    (1e300, 112, ("linear", 1e-18)), (1e8, 48, ("linear", 1e-10)), (1e20, 80, ("base", 1e100)),
])
def test_rope_tables_of_large_bases_far_out(base, R, scaling):
    """The header's bound, 2^-22 and 2^-50 of the angle, against 70 digits."""
    start, rows, amplitude = 2 ** 31 - 8, 6, 1.3
    cos, sin = (t.double().cpu() for t in AB.attn_rope_tables(rows, R, base=base, scaling=scaling, amplitude=amplitude, start=start,
                                                              device=DEV))
    with localcontext(prec=70):
        f = exact_frequencies(R, base, scaling)
        for r in range(rows):
            for i in range(R // 2):
                ang = (start + r) * f[i]
                rest = float(ang % (2 * PI))
                bound = amplitude * (2.0 ** -22 + 2.0 ** -50 * float(ang))
                assert abs(cos[r, i].item() - amplitude * math.cos(rest)) <= bound, (r, i, float(ang))
                assert abs(sin[r, i].item() - amplitude * math.sin(rest)) <= bound, (r, i, float(ang))
