"""Pins of the draft step's oracle, and the host-side refusals of its entry points (no GPU needed)."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle
from attention_attn_fwd_06_gb300 import binding as B
from attention_attn_fwd_06_gb300.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return B.load()


# ---------------------------------------------------------------- the oracle

def test_frequencies_hand_worked():
    f = oracle.rope_frequencies(16, 10000.0)
    assert np.allclose(f, 10.0 ** (-np.arange(8) / 2.0), rtol=1e-14)
    assert np.allclose(oracle.rope_frequencies(16, 10000.0, ("linear", 4.0)), f / 4, rtol=1e-14)
    # a longer base: the first pair keeps its speed, the last is slowed by the factor
    g = oracle.rope_frequencies(16, 10000.0, ("base", 4.0))
    assert g[0] == 1.0 and g[-1] == pytest.approx(f[-1] / 4, rel=1e-12) and (g[1:] < f[1:]).all()
    # turns over 1000 positions: 159, 50, 15.9, 5.03, 1.59, 0.503 ...; between 2 and 10 turns g = (t - 2) / 8
    g = oracle.rope_frequencies(16, 10000.0, ("turns", 8.0, 1000, 2.0, 10.0))
    t = 1000 * f / (2 * math.pi)
    assert np.allclose(g[:3], f[:3]) and np.allclose(g[4:], f[4:] / 8)
    assert g[3] == pytest.approx(f[3] * ((t[3] - 2) / 8 + (1 - (t[3] - 2) / 8) / 8))
    # the pair of t turns: c(10) = 8 ln(15.9) / ln(1e4) = 2.40 -> 2, c(2) = 3.80 -> 4
    g = oracle.rope_frequencies(16, 10000.0, ("index", 8.0, 1000, 2.0, 10.0))
    assert np.allclose(g[:3], f[:3]) and np.allclose(g[4:], f[4:] / 8) and g[3] == pytest.approx(f[3] * (0.5 + 0.5 / 8))


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_rotation_of_a_part(style):
    g = np.random.default_rng(1)
    x = g.normal(size=(5, 3, 64))
    cos, sin, _ = oracle.rope_table_rows(7, 5, 32)
    y, size = oracle.rotate_part(x, cos[:, None], sin[:, None], style)
    assert np.array_equal(y[..., 32:], x[..., 32:]) and (size >= np.abs(y) - 1e-12).all()
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1))  # a rotation
    whole, _ = oracle.rotate_part(x[..., :32], cos[:, None], sin[:, None], style)
    assert np.array_equal(whole, y[..., :32])
    # all of a head: the rotation that the attention calls' oracle uses (before its rounding to bf16)
    tab = [torch.from_numpy(t) for t in oracle.rope_table_rows(0, 12, 64)[:2]]
    want = oracle.rope_rotate(x[:, 0], np.arange(7, 12), *tab, style)
    full, _ = oracle.rotate_part(x[:, 0], tab[0].numpy()[7:], tab[1].numpy()[7:], style)
    assert np.allclose(oracle.round_bf16(full), want, atol=2 ** -7)


def test_pages_round_trip_and_decode():
    g = np.random.default_rng(2)
    k, v = g.normal(size=(2, 30, 2, 64))
    q = g.normal(size=(7, 4, 64))
    kp, vp = np.full((2, 9, 2, 8, 64), np.nan)
    table, slots = np.array([[4, 0, 8], [7, 2, -1]]), []
    for b, n in enumerate((17, 13)):
        slots += [int(table[b][j // 8]) * 8 + j % 8 for j in range(n)]
    oracle.append_paged(kp, k, slots)
    oracle.append_paged(vp, v, slots)
    assert np.array_equal(oracle.read_paged(kp, table[0], 17), k[:17])
    assert np.array_equal(oracle.read_paged(vp, table[1], 13), v[17:])
    assert np.isfinite(kp).all(-1).sum() == 60
    cu = [0, 3, 7]
    O, lse = oracle.decode_multi_paged(q, kp, vp, table, [17, 13], cu, 0.1)
    for b, (t0, t1, k0, k1) in enumerate(((0, 3, 0, 17), (3, 7, 17, 30))):
        dense = [np.moveaxis(x[k0:k1], 0, 1)[None] for x in (k, v)]
        o, ls = oracle.decode_multi(np.moveaxis(q[t0:t1], 0, 1)[None], *dense, [k1 - k0], 0.1)
        assert np.allclose(O[t0:t1], np.moveaxis(o[0], 1, 0)) and np.allclose(lse[t0:t1], np.moveaxis(ls[0], 1, 0))
    O, lse = oracle.decode_multi_paged(q, kp, vp, table, [2, 0], cu, 0.1)  # three tokens on two keys; none at all
    assert not O[0].any() and np.isneginf(lse[0]).all() and np.isfinite(lse[1:3]).all() and np.isneginf(lse[3:]).all()


def test_verify_hand_worked():
    p = [[0.5, 0.25, 0.25, 0.0], [0.125, 0.125, 0.5, 0.25], [0.0, 0.5, 0.0, 0.5]]
    q = [[0.25, 0.5, 0.25, 0.0], [0.25, 0.25, 0.25, 0.25]]
    # draft 1 of the first row: 0.5 q < p up to u = 0.5; then the rest is (0.25, 0, 0, 0)
    assert oracle.verify_drafts([1, 2], p, [0.5, 0.0, 0.9], q) == (0, 0)
    # stands below it; draft 2 has p > q; the last row decides: weights 0, .5, 0, .5
    assert oracle.verify_drafts([1, 2], p, [0.49, 0.99, 0.49], q) == (2, 1)
    assert oracle.verify_drafts([1, 2], p, [0.49, 0.99, 0.5], q) == (2, 3)
    # the second refused: rest (0, 0, .25, 0)
    assert oracle.verify_drafts([1, 0], p, [0.0, 0.5, 0.0], q) == (1, 2)
    # without a distribution: u < p, and the refused draft cannot come out
    assert oracle.verify_drafts([0, 2], p, [0.49, 0.6, 0.0], None) == (1, 0)
    assert oracle.verify_drafts([0, 2], p, [0.49, 0.6, 0.99], None) == (1, 3)
    assert oracle.verify_drafts([], p[:1], [0.6], None) == (0, 1)
    # p nowhere above q: p itself; no weight at all; u of 1; a token out of range
    assert oracle.verify_drafts([3], [p[0], p[1]], [0.5, 0.6], [p[0]]) == (0, 1)
    assert oracle.verify_drafts([], [[0.0, -1.0, float("nan"), float("inf")]], [0.5]) == (0, -1)
    assert oracle.verify_drafts([], p[:1], [1.0]) == (0, 2) and oracle.verify_drafts([], p[:1], [float("nan")]) == (0, 2)
    assert oracle.verify_drafts([4], [p[0], p[1]], [0.0, 0.0], [q[0]]) == (0, 0)


def test_verified_tokens_are_distributed_as_the_target():
    """Over all drafts and a fine grid of random numbers, the next token comes out with the target's probabilities."""
    p, q = [0.5, 0.125, 0.375], [0.25, 0.5, 0.25]
    n, got = 64, np.zeros(3)
    grid = [(i + 0.5) / n for i in range(n)]
    for x in range(3):
        for u in grid:
            for last in grid:
                stand, token = oracle.verify_drafts([x], [p, p], [u, last], [q])
                got[x if stand else token] += q[x] / n ** 2
    assert np.abs(got - p).max() < 1.5 / n


# ---------------------------------------------------------------- refusals

FAKE = 1 << 20


def params(cls, **kw):
    p = cls()
    for k, v in kw.items():
        setattr(p, k, v)
    return ctypes.byref(p)


TABLES = dict(cos=FAKE, sin=FAKE, rows=4, start=0, rotary_dim=64, base=1e4, factor=2.0, context=4096.0, low=1.0, high=4.0,
              amplitude=1.0)


@pytest.mark.parametrize("kw,code", [
    (dict(cos=None), B.ATTN_ERR_INVALID_ARG),
    (dict(sin=None), B.ATTN_ERR_INVALID_ARG),
    (dict(rows=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(start=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(rotary_dim=0), B.ATTN_ERR_INVALID_ARG),
    (dict(rotary_dim=24), B.ATTN_ERR_UNSUPPORTED),
    (dict(rotary_dim=144), B.ATTN_ERR_UNSUPPORTED),
    (dict(rows=2 ** 31 - 1, start=1), B.ATTN_ERR_UNSUPPORTED),
    (dict(base=1.0), B.ATTN_ERR_INVALID_ARG),
    (dict(base=float("inf")), B.ATTN_ERR_INVALID_ARG),
    (dict(amplitude=float("nan")), B.ATTN_ERR_INVALID_ARG),
    (dict(amplitude=1e300), B.ATTN_ERR_INVALID_ARG),
    (dict(scaling=5), B.ATTN_ERR_INVALID_ARG),
    (dict(scaling=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(scaling=B.ATTN_ROPE_SCALE_LINEAR, factor=0.0), B.ATTN_ERR_INVALID_ARG),
    (dict(scaling=B.ATTN_ROPE_SCALE_BASE, factor=float("nan")), B.ATTN_ERR_INVALID_ARG),
    (dict(scaling=B.ATTN_ROPE_SCALE_BASE, factor=1e-300), B.ATTN_ERR_INVALID_ARG),
    (dict(scaling=B.ATTN_ROPE_SCALE_TURNS, low=4.0), B.ATTN_ERR_INVALID_ARG),
    (dict(scaling=B.ATTN_ROPE_SCALE_INDEX, low=0.0), B.ATTN_ERR_INVALID_ARG),
    (dict(scaling=B.ATTN_ROPE_SCALE_INDEX, context=0.0), B.ATTN_ERR_INVALID_ARG),
    (dict(cos=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
])
def test_rope_tables_refusals(lib, kw, code):
    assert lib.attn_rope_tables(params(B.attn_rope_tables_params, **{**TABLES, **kw})) == code


APPEND = dict(k=FAKE, v=FAKE, kpages=FAKE, vpages=FAKE, slots=FAKE, positions=FAKE, q=FAKE, q_out=FAKE, k_out=FAKE, T=2, Hq=4,
              Hkv=2, D=128, page_size=16, num_pages=4, rotary_dim=64,
              **{f"{t}_{axis}_stride": n for t in ("k", "v", "q", "q_out", "k_out") for axis, n in (("token", 512), ("head", 128))},
              rope_cos=FAKE, rope_sin=FAKE, rope_max_pos=16, rope_style=B.ATTN_ROPE_HALF)
NO_ROPE = dict(rope_style=B.ATTN_ROPE_NONE, q=None, q_out=None, k_out=None, Hq=0)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), B.ATTN_ERR_INVALID_ARG),
    (dict(vpages=None), B.ATTN_ERR_INVALID_ARG),
    (dict(slots=None), B.ATTN_ERR_INVALID_ARG),
    (dict(positions=None), B.ATTN_ERR_INVALID_ARG),
    (dict(q=None), B.ATTN_ERR_INVALID_ARG),
    (dict(q=None, q_out=None), B.ATTN_ERR_INVALID_ARG),
    (dict(Hq=0), B.ATTN_ERR_INVALID_ARG),
    (dict(Hq=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(Hkv=0), B.ATTN_ERR_INVALID_ARG),
    (dict(T=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(page_size=0), B.ATTN_ERR_INVALID_ARG),
    (dict(num_pages=0), B.ATTN_ERR_INVALID_ARG),
    (dict(rotary_dim=0), B.ATTN_ERR_INVALID_ARG),
    (dict(rotary_dim=40), B.ATTN_ERR_UNSUPPORTED),
    (dict(rotary_dim=144), B.ATTN_ERR_UNSUPPORTED),
    (dict(D=96), B.ATTN_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 28), B.ATTN_ERR_UNSUPPORTED),
    (dict(Hq=65535), B.ATTN_ERR_UNSUPPORTED),
    (dict(rope_style=3), B.ATTN_ERR_INVALID_ARG),
    (dict(rope_sin=None), B.ATTN_ERR_INVALID_ARG),
    (dict(rope_max_pos=0), B.ATTN_ERR_INVALID_ARG),
    (dict(NO_ROPE, k_out=FAKE), B.ATTN_ERR_INVALID_ARG),
    (dict(NO_ROPE, q=FAKE, q_out=FAKE, Hq=4), B.ATTN_ERR_INVALID_ARG),
    (dict(kpages=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(q_out=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
    (dict(v_head_stride=132), B.ATTN_ERR_ALIGNMENT),
    (dict(q_token_stride=260), B.ATTN_ERR_ALIGNMENT),
    (dict(k_out_token_stride=260), B.ATTN_ERR_ALIGNMENT),
    (dict(slots=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
])
def test_kv_append_paged_refusals(lib, kw, code):
    assert lib.attn_kv_append_paged(params(B.attn_kv_append_paged_params, **{**APPEND, **kw})) == code


DECODE = dict(q=FAKE, kpages=FAKE, vpages=FAKE, block_table=FAKE, kv_lens=FAKE, cu_new=FAKE, out=FAKE, lse=FAKE, B=2, T=8, Hq=8,
              Hkv=2, D=128, max_new=4, page_size=16, max_pages=4, num_pages=8, scale=0.1)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.ATTN_ERR_INVALID_ARG),
    (dict(cu_new=None), B.ATTN_ERR_INVALID_ARG),
    (dict(block_table=None), B.ATTN_ERR_INVALID_ARG),
    (dict(out=None), B.ATTN_ERR_INVALID_ARG),
    (dict(B=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(T=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(Hq=9), B.ATTN_ERR_INVALID_ARG),
    (dict(max_new=0), B.ATTN_ERR_INVALID_ARG),
    (dict(max_new=33), B.ATTN_ERR_UNSUPPORTED),
    (dict(D=96), B.ATTN_ERR_UNSUPPORTED),
    (dict(page_size=4), B.ATTN_ERR_INVALID_ARG),
    (dict(page_size=12), B.ATTN_ERR_UNSUPPORTED),
    (dict(max_pages=0), B.ATTN_ERR_INVALID_ARG),
    (dict(max_pages=1 << 27), B.ATTN_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 30), B.ATTN_ERR_UNSUPPORTED),
    (dict(T=1 << 28), B.ATTN_ERR_UNSUPPORTED),
    (dict(B=32767 + 1), B.ATTN_ERR_UNSUPPORTED),
    (dict(scale=float("nan")), B.ATTN_ERR_INVALID_ARG),
    (dict(out_dtype=2), B.ATTN_ERR_INVALID_ARG),
    (dict(kpages=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(workspace=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(cu_new=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
])
def test_decode_multi_paged_refusals(lib, kw, code):
    assert lib.attn_decode_multi_paged(params(B.attn_decode_multi_paged_params, **{**DECODE, **kw})) == code


VERIFY = dict(draft_tokens=FAKE, target_probs=FAKE, draft_probs=FAKE, uniforms=FAKE, draft_lens=FAKE, kv_lens=FAKE, tokens=FAKE,
              accepted=FAKE, keep_lens=FAKE, B=2, K=3, V=100, dtype=B.ATTN_DTYPE_F32, target_sequence_stride=400,
              target_row_stride=100, draft_sequence_stride=300, draft_row_stride=100)


@pytest.mark.parametrize("kw,code", [
    (dict(draft_tokens=None), B.ATTN_ERR_INVALID_ARG),
    (dict(target_probs=None), B.ATTN_ERR_INVALID_ARG),
    (dict(target_probs=None, cu_target=FAKE, total=1), B.ATTN_ERR_INVALID_ARG),
    (dict(uniforms=None), B.ATTN_ERR_INVALID_ARG),
    (dict(tokens=None), B.ATTN_ERR_INVALID_ARG),
    (dict(accepted=None), B.ATTN_ERR_INVALID_ARG),
    (dict(kv_lens=None), B.ATTN_ERR_INVALID_ARG),
    (dict(keep_lens=None), B.ATTN_ERR_INVALID_ARG),
    (dict(B=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(K=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(V=0), B.ATTN_ERR_INVALID_ARG),
    (dict(cu_target=FAKE, total=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(dtype=2), B.ATTN_ERR_INVALID_ARG),
    (dict(K=1 << 20), B.ATTN_ERR_UNSUPPORTED),
    (dict(V=1 << 30), B.ATTN_ERR_UNSUPPORTED),
    (dict(B=1 << 26), B.ATTN_ERR_UNSUPPORTED),
    (dict(target_probs=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
    (dict(dtype=B.ATTN_DTYPE_BF16, draft_probs=FAKE + 1), B.ATTN_ERR_ALIGNMENT),
    (dict(uniforms=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
    (dict(keep_lens=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
])
def test_verify_drafts_refusals(lib, kw, code):
    assert lib.attn_verify_drafts(params(B.attn_verify_drafts_params, **{**VERIFY, **kw})) == code


def test_empty_calls_succeed_without_a_device(lib):
    assert lib.attn_rope_tables(params(B.attn_rope_tables_params, **{**TABLES, "rows": 0})) == B.ATTN_OK
    assert lib.attn_kv_append_paged(params(B.attn_kv_append_paged_params, **{**APPEND, "T": 0})) == B.ATTN_OK
    assert lib.attn_decode_multi_paged(params(B.attn_decode_multi_paged_params, **{**DECODE, "B": 0})) == B.ATTN_OK
    assert lib.attn_decode_multi_paged(params(B.attn_decode_multi_paged_params, **{**DECODE, "T": 0})) == B.ATTN_OK
    assert lib.attn_verify_drafts(params(B.attn_verify_drafts_params, **{**VERIFY, "B": 0})) == B.ATTN_OK


def test_calls_fail_without_a_device(lib):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    no_device = (B.ATTN_ERR_UNSUPPORTED, B.ATTN_ERR_CUDA)
    for fn, cls, kw in ((lib.attn_rope_tables, B.attn_rope_tables_params, TABLES),
                        (lib.attn_kv_append_paged, B.attn_kv_append_paged_params, APPEND),
                        (lib.attn_kv_append_paged, B.attn_kv_append_paged_params, {**APPEND, **NO_ROPE, "positions": None}),
                        (lib.attn_decode_multi_paged, B.attn_decode_multi_paged_params, DECODE),
                        (lib.attn_verify_drafts, B.attn_verify_drafts_params, VERIFY),
                        (lib.attn_verify_drafts, B.attn_verify_drafts_params, {**VERIFY, "K": 0, "draft_tokens": None})):
        assert fn(params(cls, **kw)) in no_device
    # strides of axes of one element are not looked at
    one = {f"{t}_token_stride": 3 for t in ("k", "v", "q", "q_out", "k_out")}
    assert lib.attn_kv_append_paged(params(B.attn_kv_append_paged_params, **{**APPEND, **one, "T": 1})) in no_device


def test_parameter_structs_match_the_header(tmp_path):
    """Offsets of the last field and sizes of the ctypes mirrors against a C compiler's view of the header."""
    names = ["attn_rope_tables_params", "attn_kv_append_paged_params", "attn_decode_multi_paged_params",
             "attn_verify_drafts_params"]
    src = tmp_path / "sizes.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "attn.h"\nint main(void) {\n' + "".join(
        f'  printf("%zu %zu\\n", sizeof({n}), offsetof({n}, stream));\n' for n in names) + "  return 0;\n}\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "sizes")],
                   check=True)
    out = subprocess.run([str(tmp_path / "sizes")], check=True, capture_output=True, text=True).stdout.split()
    want = [x for n in names for x in (ctypes.sizeof(getattr(B, n)), getattr(B, n).stream.offset)]
    assert [int(x) for x in out] == want


def test_sizes(lib):
    small, large = (B.attn_decode_multi_paged_workspace_bytes(8, 2, n, 128) for n in (1, 32))
    assert 0 < small < large
    assert B.attn_decode_multi_paged_workspace_bytes(8, 2, 33, 128) == 0
    assert B.attn_decode_multi_paged_workspace_bytes(8, 3, 1, 128) == 0


def test_binding_refuses_what_the_kernels_would_misread():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    pool = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.attn_kv_append_paged(x, x, pool, pool, i)
    with pytest.raises(TypeError):
        B.attn_kv_append_paged(x.float(), x, pool, pool, i)
    with pytest.raises(ValueError, match="CUDA"):
        B.attn_decode_multi_paged(x, pool, pool, i[None], i, i, 1)
    with pytest.raises(ValueError, match="CUDA"):
        B.attn_verify_drafts(i[None], torch.zeros(1, 5, 7), torch.zeros(1, 5))
    with pytest.raises(ValueError, match="scaling"):
        B.attn_rope_tables(4, 64, scaling=("cubic", 2.0))
    with pytest.raises(ValueError, match="numbers"):
        B.attn_rope_tables(4, 64, scaling=("turns", 2.0))
    with pytest.raises(ValueError):
        B.attn_rope_tables(4, 63)
