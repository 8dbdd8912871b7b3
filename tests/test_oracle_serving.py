"""Pins of the serving-step oracle, and the host-side refusals of the serving-step entry points (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from attention_attn_fwd_06_gb300 import binding as B
from attention_attn_fwd_06_gb300.build import build
from tests._serving import decode_bound, make_pool, make_table


@pytest.fixture(scope="module")
def lib():
    build()
    return B.load()


def test_page_step_hand_worked():
    # pages of 4: row 0 has 5 keys (pages 7, 2), row 1 none, row 2 has 8 (pages 0, 4)
    lens, table, stack = [5, 0, 8], [[7, 2, -1], [-1, -1, -1], [0, 4, -1]], [9, 6, 5, 3]
    got = oracle.page_step(lens, table, stack, 4, 4, new_lens=[3, 2, 1])
    assert got[0] == [8, 2, 9] and got[1] == [[7, 2, -1], [3, -1, -1], [0, 4, 5]] and got[2] == [9, 6]
    assert got[3] == [9, 10, 11, 12, 13, 20] and got[4] == [5, 6, 7, 0, 1, 8] and got[5] == [0, 3, 5, 6]
    back = oracle.page_step(got[0], got[1], got[2], 2, 4, keep_lens=lens)
    assert back[0] == lens and back[1] == table and back[2] == stack
    assert oracle.page_step(lens, table, stack, 1, 4, new_lens=[3, 2, 1]) is None       # one page, two wanted
    assert oracle.page_step(lens, table, stack, 4, 4, new_lens=[8, 0, 0]) is None       # row of more than 3 pages
    assert oracle.page_step(lens, table, stack, 4, 4, keep_lens=[6, 0, 0]) is None      # more kept than there is
    swap = oracle.page_step(lens, table, [], 0, 4, keep_lens=[0, 0, 8], new_lens=[0, 8, 0])
    assert swap[1] == [[-1, -1, -1], [7, 2, -1], [0, 4, -1]] and swap[2] == []         # given back and taken at once


def test_quantise_hand_worked_and_round_trip():
    x = np.zeros((1, 64))
    x[0, :4] = [-1.0, 14.0, 2.5, 1.5]
    u, s, m = oracle.quantise_q4(x)
    assert s[0, 0] == 1.0 and m[0, 0] == -1.0 and u[0, 0, :5].tolist() == [0, 15, 4, 2, 1]  # 3.5 and 2.5: ties to even
    assert np.array_equal(oracle.values_q4(u, s, m)[0, :5], [-1, 14, 3, 1, 0])
    u, s, m = oracle.quantise_q4(np.full((1, 64), 3.0))
    assert s[0, 0] == 0 and not u.any() and m[0, 0] == 3.0
    u, s, m = oracle.quantise_q4(np.array([[np.nan, np.inf, -np.inf] + [0.0] * 61]))
    assert m[0, 0] == -65504 and oracle.values_q4(u, s, m)[0, 1] == pytest.approx(65504, rel=1e-3)
    x = np.random.default_rng(1).normal(size=(50, 3, 128))
    u, s, m = oracle.quantise_q4(x)
    # a code is half a step off at most, and scale and minimum are rounded to 11 bits
    err = np.abs(oracle.values_q4(u, s, m) - x).reshape(50, 3, 2, 64)
    assert (err <= 0.5 * s[..., None] + 2.0 ** -11 * (np.abs(m) + 15 * s)[..., None]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_pool_round_trip(D):
    g = np.random.default_rng(D)
    pool = make_pool(5, 2, 48, D, 1, poison=True)
    table, _ = make_table([100], 48, 5, 2)
    pos = np.arange(100)
    slots = table[0][pos // 48] * 48 + pos % 48
    k, v = g.normal(size=(2, 100, 2, D))
    oracle.write_q4(pool, k, v, slots)
    kk, vv, kt, vt = oracle.read_q4(pool, table[0], 10, 100)
    for got, term, x in ((kk, kt, k), (vv, vt, v)):
        want = oracle.values_q4(*oracle.quantise_q4(x))[10:]
        assert np.array_equal(got, want) and (np.abs(got) <= term).all()


def test_decode_reference_agrees_with_decode_multi():
    pool = make_pool(8, 2, 16, 64, 3)
    table, _ = make_table([33, 7], 16, 8, 4)
    q = torch.randn(2, 4, 3, 64, dtype=torch.float64)
    O, lse, _, _ = decode_bound(q, pool, table, [33, 7], 0.2, False)
    for b, n in enumerate((33, 7)):
        k, v, _, _ = oracle.read_q4(pool, table[b], 0, n)
        Or, lr = oracle.decode_multi(q[b:b + 1], k.transpose(1, 0, 2)[None], v.transpose(1, 0, 2)[None], [n], 0.2)
        assert np.allclose(O[b], Or[0]) and np.allclose(lse[b], lr[0])


def test_rms_norm_closed_form():
    x = np.array([[3.0, 4.0] * 32])
    assert np.allclose(oracle.rms_norm(x, None, 0.0), x / np.sqrt(12.5))
    assert np.allclose(oracle.rms_norm(x, np.full(64, 2.0), 12.5), 2 * x / 5)


FAKE = 1 << 20  # 128-byte aligned, never dereferenced: validation happens first


def params(cls, **kw):
    p = cls()
    for k, v in kw.items():
        setattr(p, k, v)
    return ctypes.byref(p)


PAGE = dict(kv_lens=FAKE, block_table=FAKE, free_pages=FAKE, free_count=FAKE, B=2, page_size=16, max_pages=4,
            num_pages=8, max_tokens=4)


@pytest.mark.parametrize("kw,code", [
    (dict(kv_lens=None), B.ATTN_ERR_INVALID_ARG),
    (dict(block_table=None), B.ATTN_ERR_INVALID_ARG),
    (dict(free_pages=None), B.ATTN_ERR_INVALID_ARG),
    (dict(free_count=None), B.ATTN_ERR_INVALID_ARG),
    (dict(B=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(page_size=0), B.ATTN_ERR_INVALID_ARG),
    (dict(max_pages=0), B.ATTN_ERR_INVALID_ARG),
    (dict(num_pages=0), B.ATTN_ERR_INVALID_ARG),
    (dict(max_tokens=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(B=8193), B.ATTN_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 28), B.ATTN_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 28), B.ATTN_ERR_UNSUPPORTED),
    (dict(slots=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
    (dict(cu_new=FAKE + 1), B.ATTN_ERR_ALIGNMENT),
])
def test_page_step_refusals(lib, kw, code):
    assert lib.attn_page_step(params(B.attn_page_step_params, **{**PAGE, **kw})) == code


NORM = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, positions=FAKE, B=1, L=4, Hq=4, Hkv=2, D=128, eps=1e-6,
            **{f"{t}_{axis}_stride": n for t in ("q", "k", "q_out", "k_out") for axis, n in
               (("sequence", 0), ("token", 512), ("head", 128))},
            rope_cos=FAKE, rope_sin=FAKE, rope_max_pos=16, rope_style=B.ATTN_ROPE_HALF)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.ATTN_ERR_INVALID_ARG),
    (dict(k_out=None), B.ATTN_ERR_INVALID_ARG),
    (dict(positions=None), B.ATTN_ERR_INVALID_ARG),
    (dict(Hq=0), B.ATTN_ERR_INVALID_ARG),
    (dict(L=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(eps=-1e-6), B.ATTN_ERR_INVALID_ARG),
    (dict(eps=float("nan")), B.ATTN_ERR_INVALID_ARG),
    (dict(rope_style=9), B.ATTN_ERR_INVALID_ARG),
    (dict(rope_sin=None), B.ATTN_ERR_INVALID_ARG),
    (dict(D=96), B.ATTN_ERR_UNSUPPORTED),
    (dict(B=1 << 16, L=1 << 16), B.ATTN_ERR_UNSUPPORTED),
    (dict(q=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(k_weight=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
    (dict(q_head_stride=132), B.ATTN_ERR_ALIGNMENT),
    (dict(k_out_token_stride=260), B.ATTN_ERR_ALIGNMENT),
    (dict(positions=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
])
def test_qk_norm_rope_refusals(lib, kw, code):
    assert lib.attn_qk_norm_rope(params(B.attn_qk_norm_rope_params, **{**NORM, **kw})) == code


APPEND = dict(k=FAKE, v=FAKE, pool=FAKE, slots=FAKE, T=2, Hkv=2, D=128, page_size=16, num_pages=4,
              k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128)


@pytest.mark.parametrize("kw,code", [
    (dict(v=None), B.ATTN_ERR_INVALID_ARG),
    (dict(pool=None), B.ATTN_ERR_INVALID_ARG),
    (dict(T=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(page_size=24), B.ATTN_ERR_INVALID_ARG),
    (dict(page_size=8), B.ATTN_ERR_INVALID_ARG),
    (dict(num_pages=0), B.ATTN_ERR_INVALID_ARG),
    (dict(Hkv=0), B.ATTN_ERR_INVALID_ARG),
    (dict(D=32), B.ATTN_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 28), B.ATTN_ERR_UNSUPPORTED),
    (dict(pool=FAKE + 64), B.ATTN_ERR_ALIGNMENT),
    (dict(k_head_stride=4), B.ATTN_ERR_ALIGNMENT),
    (dict(slots=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
])
def test_kv_append_refusals(lib, kw, code):
    assert lib.attn_kv_append_q4(params(B.attn_kv_append_q4_params, **{**APPEND, **kw})) == code


GATHER = dict(pool=FAKE, block_table=FAKE, cu_k=FAKE, k=FAKE, v=FAKE, B=1, Hkv=2, D=64, page_size=16, max_pages=4,
              num_pages=4, total_k=8)


@pytest.mark.parametrize("kw,code", [
    (dict(cu_k=None), B.ATTN_ERR_INVALID_ARG),
    (dict(k=None), B.ATTN_ERR_INVALID_ARG),
    (dict(total_k=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(max_pages=0), B.ATTN_ERR_INVALID_ARG),
    (dict(max_pages=1 << 28), B.ATTN_ERR_UNSUPPORTED),
    (dict(v=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(kv_starts=FAKE + 1), B.ATTN_ERR_ALIGNMENT),
])
def test_kv_gather_refusals(lib, kw, code):
    assert lib.attn_kv_gather_q4(params(B.attn_kv_gather_q4_params, **{**GATHER, **kw})) == code


DECODE = dict(q=FAKE, pool=FAKE, block_table=FAKE, kv_lens=FAKE, out=FAKE, B=2, Hq=8, Hkv=2, Lq=1, D=128, page_size=16,
              max_pages=4, num_pages=8, scale=0.1)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.ATTN_ERR_INVALID_ARG),
    (dict(block_table=None), B.ATTN_ERR_INVALID_ARG),
    (dict(Hq=7), B.ATTN_ERR_INVALID_ARG),
    (dict(Lq=0), B.ATTN_ERR_INVALID_ARG),
    (dict(chunk=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(out_dtype=3), B.ATTN_ERR_INVALID_ARG),
    (dict(scale=float("inf")), B.ATTN_ERR_INVALID_ARG),
    (dict(page_size=20), B.ATTN_ERR_INVALID_ARG),
    (dict(Lq=33), B.ATTN_ERR_UNSUPPORTED),
    (dict(D=256), B.ATTN_ERR_UNSUPPORTED),
    (dict(max_pages=1 << 27), B.ATTN_ERR_UNSUPPORTED),
    (dict(out=FAKE + 4), B.ATTN_ERR_ALIGNMENT),
    (dict(workspace=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(pool=FAKE + 16), B.ATTN_ERR_ALIGNMENT),
])
def test_decode_q4_refusals(lib, kw, code):
    assert lib.attn_decode_q4(params(B.attn_decode_q4_params, **{**DECODE, **kw})) == code


def test_strides_of_axes_of_one_element_are_not_looked_at(lib):
    """Whether a call is refused before it looks for a device."""
    def refused(fn, cls, base, **kw):
        return fn(params(cls, **{**base, **kw})) == B.ATTN_ERR_ALIGNMENT

    norm = lib.attn_qk_norm_rope, B.attn_qk_norm_rope_params, {**NORM, "B": 1, "L": 1}
    append = lib.attn_kv_append_q4, B.attn_kv_append_q4_params, {**APPEND, "T": 1}
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    for t in ("q", "k", "q_out", "k_out"):
        assert not refused(*norm, **{f"{t}_token_stride": 3, f"{t}_sequence_stride": 1})
        assert refused(*norm, L=2, **{f"{t}_token_stride": 3})
        assert refused(*norm, B=2, **{f"{t}_sequence_stride": 3})
        assert refused(*norm, Hq=2, Hkv=2, **{f"{t}_head_stride": 3})
    for t in ("k", "v"):
        assert not refused(*append, **{f"{t}_token_stride": 3})
        assert refused(*append, T=2, **{f"{t}_token_stride": 3})
        assert not refused(*append, Hkv=1, **{f"{t}_head_stride": 3})


def test_empty_calls_succeed_without_a_device(lib):
    assert lib.attn_page_step(params(B.attn_page_step_params, **{**PAGE, "B": 0})) == B.ATTN_OK
    assert lib.attn_qk_norm_rope(params(B.attn_qk_norm_rope_params, **{**NORM, "L": 0})) == B.ATTN_OK
    assert lib.attn_kv_append_q4(params(B.attn_kv_append_q4_params, **{**APPEND, "T": 0})) == B.ATTN_OK
    assert lib.attn_kv_gather_q4(params(B.attn_kv_gather_q4_params, **{**GATHER, "total_k": 0})) == B.ATTN_OK
    assert lib.attn_decode_q4(params(B.attn_decode_q4_params, **{**DECODE, "B": 0})) == B.ATTN_OK


def test_parameter_structs_match_the_header(tmp_path):
    """Offsets of the last field and sizes of the ctypes mirrors against a C compiler's view of the header."""
    import os
    import subprocess
    names = ["attn_page_step_params", "attn_qk_norm_rope_params", "attn_kv_append_q4_params",
             "attn_kv_gather_q4_params", "attn_decode_q4_params"]
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
    assert B.attn_kv_q4_page_bytes(16, 8, 128) == 8 * 2304 and B.attn_kv_q4_page_bytes(64, 2, 64) == 2 * 4 * 1152
    assert B.attn_kv_q4_page_bytes(24, 8, 128) == 0 and B.attn_kv_q4_page_bytes(16, 8, 80) == 0
    assert B.attn_decode_q4_workspace_bytes(32, 8, 1, 128) > 3 * 8 * 128 * 4
    assert B.attn_decode_q4_workspace_bytes(32, 8, 33, 128) == 0


def test_calls_fail_without_a_device(lib):
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    for fn, cls, kw in ((lib.attn_page_step, B.attn_page_step_params, PAGE),
                        (lib.attn_qk_norm_rope, B.attn_qk_norm_rope_params, NORM),
                        (lib.attn_kv_append_q4, B.attn_kv_append_q4_params, APPEND),
                        (lib.attn_kv_gather_q4, B.attn_kv_gather_q4_params, GATHER),
                        (lib.attn_decode_q4, B.attn_decode_q4_params, DECODE)):
        assert fn(params(cls, **kw)) in (B.ATTN_ERR_UNSUPPORTED, B.ATTN_ERR_CUDA)


def test_binding_refuses_what_the_kernels_would_misread():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.attn_qk_norm_rope(x, None)
    with pytest.raises(TypeError):
        B.attn_qk_norm_rope(x.float(), None)
    with pytest.raises(TypeError):
        B.attn_page_step([1], x, x, x, 16)
    with pytest.raises(ValueError, match="overlap"):
        B._written_once(torch.zeros(1, 2, 128).expand(4, 2, 128), "q_out")
    B._written_once(torch.zeros(4, 6, 128)[:, 2:4], "q_out")
    B._written_once(torch.zeros(2, 3, 5, 128).transpose(1, 2), "q_out")
